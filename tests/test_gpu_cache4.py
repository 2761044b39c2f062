"""The 4-bit paged cache on the GPU against its plain reference: bytes written,
values read back, attention of single tokens, a few, and chunks; slots that no
sequence holds are filled with NaN parameters throughout."""
import numpy as np
import pytest
import torch

from cache4_reference import Layout, attention, from16, quantise, to16, values

pytestmark = pytest.mark.gpu

NP16 = {torch.float16: False, torch.bfloat16: True}


@pytest.fixture(scope="module")
def c4():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from kv_cache_compression_cg_gb300 import build, cache4
    build.build()
    return cache4


def cuda16(x, dtype):
    """binary32 numpy -> 16-bit tensor on the GPU."""
    return torch.from_numpy(np.ascontiguousarray(to16(x, NP16[dtype])).view(np.int16)).cuda().view(dtype)


def host16(t):
    """16-bit tensor -> binary32 numpy."""
    return from16(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), NP16[t.dtype])


class Problem:
    """Sequences of given (tokens, rows), K and V rows of all their tokens, a pool of
    poisoned pages and a shuffled table."""

    def __init__(self, c4, seqs, L=1, P=16, H=2, D=128, group=64, dtype=torch.float16, seed=0, spare=2, scale_v=1.0):
        self.rng = rng = np.random.default_rng(seed)
        self.seqs, self.L, self.P, self.H, self.D, self.group, self.dtype, self.bf16 = seqs, L, P, H, D, group, dtype, NP16[dtype]
        need = [-(-n // P) for n, _ in seqs]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(seqs), max(need + [1]) + 1), 2 ** 31 - 1, np.int32)  # entries past a sequence's pages are never followed
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lay = Layout(L, self.pages, P, H, D, group)
        self.lens = np.array([n for n, _ in seqs], np.int32)
        self.start = np.concatenate([[0], np.cumsum([r for _, r in seqs])]).astype(np.int32)
        n = int(self.lens.sum())
        off = rng.standard_normal((H, D)) * 0.7
        k = rng.standard_normal((L, n, H, D)) * np.exp(0.5 * rng.standard_normal((H, D))) + off
        v = rng.standard_normal((L, n, H, D)) * scale_v
        self.k, self.v = (from16(to16(x.astype(np.float32), self.bf16), self.bf16) for x in (k, v))
        self.cache = c4.Cache4(L, self.pages, P, H, D, group=group, dtype=dtype)
        self.cache.pool.fill_(0xFF)
        self.c4 = c4

    def batch(self, rows=None, **kw):
        start = torch.from_numpy(self.start).cuda() if rows is None else torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32).cuda()
        n = [r for _, r in self.seqs] if rows is None else rows
        return self.c4.Batch4(torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda(), start,
                              rows=int(sum(n)), max_rows=int(max(list(n) + [0])), **kw)

    def fill(self):
        """All tokens of all sequences into the pool, through write_layers."""
        k, v = (cuda16(x.reshape(self.L, -1, self.H * self.D), self.dtype) for x in (self.k, self.v))
        self.cache.write_layers(k, v, self.batch(list(self.lens)))
        return self

    def token(self, b, j):
        return int(self.lens[:b].sum()) + j

    def slot(self, b, j):
        return int(self.table[b, j // self.P]), j % self.P

    def flags(self):
        torch.cuda.synchronize()
        return int(self.cache.status.item())


STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def check_attention(pr, q, out, lse, window=0, scale=None, sample=None, layer=0, hidden=()):
    """Every (row, head), or a sample of them. hidden: (sequence, page index) that no query sees."""
    torch.cuda.synchronize()
    out, q = host16(out).astype(np.float64), host16(q).astype(np.float64)
    lse = None if lse is None else lse.cpu().numpy().astype(np.float64)
    Hq, D, H, G = q.shape[1], pr.D, pr.H, pr.group
    scale = D ** -0.5 if scale is None else scale
    tables = {}
    for x, name in ((pr.k[layer], "k"), (pr.v[layer], "v")):
        c, p = quantise(x, G, pr.bf16)
        f = from16(p, pr.bf16).astype(np.float64)
        tables[name] = values(c, p, G, pr.bf16).astype(np.float64)  # s c + m fits binary64; U's rounding is within the bound's u
        tables[name + "t"] = np.repeat(15 * f[..., 0] + np.abs(f[..., 1]), G, -1)
    todo = [(b, i, h) for b, (n, r) in enumerate(pr.seqs) for i in range(r) for h in range(Hq)]
    if sample and len(todo) > sample:
        keep = set(pr.rng.choice(len(todo), sample, replace=False).tolist()) | {0, len(todo) - 1}
        todo = [t for i, t in enumerate(todo) if i in keep]
    for b, i, h in todo:
        n, r = pr.seqs[b]
        row, kvh = int(pr.start[b]) + i, h // (Hq // H)
        rows = np.arange(pr.token(b, 0), pr.token(b, 0) + n)
        j = np.arange(n)
        drop = np.isin(j // pr.P, [pg for s, pg in hidden if s == b])
        k, v, t = (tables[x][rows, kvh] for x in ("k", "v", "kt"))
        pos = n - r + i
        if drop.any():
            assert not window
            vis = ~drop & (j <= pos)
            k, v, t, pos = k[vis], v[vis], t[vis], vis.sum() - 1
        want, wl, bound, bl = attention(q[row, h], k, v, pos, window, scale, t, STEP[pr.dtype])
        got = out[row, h]
        nan = np.isnan(want)  # channels of a value group that is not finite
        assert np.array_equal(np.isnan(got), nan), (b, i, h, np.isnan(got).sum(), nan.sum())
        assert (np.abs(got - want) <= bound)[~nan].all(), (b, i, h, float(np.nanmax(np.abs(got - want) / bound)))
        if lse is not None:
            if np.isneginf(wl):
                assert np.isneginf(lse[row, h])
            else:
                assert abs(lse[row, h] - wl) <= bl, (b, i, h, lse[row, h], wl, bl)


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,group", SHAPES)
def test_write_bytes_and_read_values(c4, D, group, dtype):
    """Each written token's codes and parameters bit for bit, no other byte touched, values read back exactly."""
    pr = Problem(c4, [(37, 5), (1, 1), (16, 16), (0, 0), (83, 20)], L=2, P=32, H=3, D=D, group=group, dtype=dtype)
    b = pr.batch()
    rows = [pr.token(s, n - r + i) for s, (n, r) in enumerate(pr.seqs) for i in range(r)]
    k, v = (cuda16(x[:, rows].reshape(2, len(rows), -1), dtype) for x in (pr.k, pr.v))
    pr.cache.write_layers(k, v, b)
    assert pr.flags() == 0
    want = np.full(pr.lay.nbytes, 0xFF, np.uint8)
    for layer in range(2):
        for x, is_v in ((pr.k, False), (pr.v, True)):
            c, p = quantise(x[layer], group, pr.bf16)
            for s, (n, r) in enumerate(pr.seqs):
                for i in range(r):
                    t = pr.token(s, n - r + i)
                    page, slot = pr.slot(s, n - r + i)
                    for h in range(3):
                        pr.lay.put(want, layer, page, h, slot, is_v, c[t, h], p[t, h])
    got = pr.cache.pool.cpu().numpy().reshape(-1)
    assert np.array_equal(got, want)
    for out in (None, torch.float32):
        rk, rv = pr.cache.read_layers(b, dtype=out)
        torch.cuda.synchronize()
        for x, y in ((pr.k, rk), (pr.v, rv)):
            for layer in range(2):
                c, p = quantise(x[layer][rows], group, pr.bf16)
                ref = values(c, p, group, pr.bf16).reshape(len(rows), -1)
                have = y[layer].cpu().numpy() if out else y[layer].view(torch.int16).cpu().numpy().view(np.uint16)
                assert np.array_equal(have, ref if out else to16(ref, pr.bf16))


@pytest.mark.parametrize("D,pad", [(64, 8), (128, 3), (256, 1)])
def test_rows_of_a_wider_tensor(c4, D, pad):
    """K and V sliced out of wider rows, aligned or not, and outputs into wider rows."""
    pr = Problem(c4, [(9, 9), (30, 13)], H=2, D=D, group=32, dtype=torch.bfloat16)
    rows = [pr.token(s, n - r + i) for s, (n, r) in enumerate(pr.seqs) for i in range(r)]
    wide = torch.full((len(rows), 5 * 2 * D + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = wide[:, pad:pad + 2 * D], wide[:, 2 * D + pad:4 * D + pad]
    k.copy_(cuda16(pr.k[0][rows].reshape(len(rows), -1), pr.dtype))
    v.copy_(cuda16(pr.v[0][rows].reshape(len(rows), -1), pr.dtype))
    b = pr.batch()
    pr.cache.write(k, v, b)
    plain = pr.cache.read(b)
    out = torch.full((2, len(rows), 2 * D + pad), 3.0, dtype=torch.float32, device="cuda")
    o = [out[i, :, pad:].unflatten(1, (2, D)) for i in range(2)]
    pr.cache.read(b, dtype=torch.float32, out=o)
    assert pr.flags() == 0
    for x, y, z in zip((pr.k, pr.v), plain, o):
        c, p = quantise(x[0][rows], 32, True)
        ref = values(c, p, 32, True)
        assert np.array_equal(z.cpu().numpy(), ref)
        assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), to16(ref, True))
    assert (out[:, :, :pad] == 3.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_extreme_values(c4, dtype):
    """Constant groups, subnormals, the type's largest values, infinities and NaNs."""
    big = 65504.0 if dtype == torch.float16 else 3.3895e38
    tiny = 6e-8 if dtype == torch.float16 else 1e-40
    x = np.zeros((9, 1, 64), np.float32)
    x[1] = -3.25
    x[2, 0, ::2] = big
    x[3, 0, ::3], x[3, 0, 1::3] = big / 4, -big / 4
    x[4, 0, :7] = tiny
    x[5] = np.linspace(-1e-6, 3e-6, 64) if dtype == torch.float16 else np.linspace(-1e-39, 3e-39, 64)
    x[6, 0, 5] = np.inf
    x[7, 0, 40] = np.nan
    x[8, 0, :32], x[8, 0, 32:] = -np.inf, 2.0
    x = from16(to16(x, NP16[dtype]), NP16[dtype])
    cache = c4.Cache4(1, 1, 16, 1, 64, group=32, dtype=dtype)
    b = c4.Batch4(torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([9], dtype=torch.int32).cuda(),
                  torch.tensor([0, 9], dtype=torch.int32).cuda(), rows=9)
    t = cuda16(x, dtype)
    cache.write(t[:6], t[:6].flip(0), c4.Batch4(b.table, torch.tensor([6], dtype=torch.int32).cuda(),
                                                torch.tensor([0, 6], dtype=torch.int32).cuda(), rows=6))
    assert int(cache.status.item()) == 0
    cache.write(t, t.flip(0), b)
    from kv_cache_compression_cg_gb300 import capi
    assert int(cache.status.item()) == capi.CG_FLAG_NONFINITE
    c, p = quantise(x, 32, NP16[dtype])
    ref = values(c, p, 32, NP16[dtype])
    k, v = cache.read(b, dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy(), ref, equal_nan=True)
    assert np.array_equal(v.cpu().numpy(), ref[::-1], equal_nan=True)
    k, v = cache.read(b)
    most = 65504.0 if dtype == torch.float16 else 3.3895313892515355e38
    with np.errstate(invalid="ignore"):
        lim = to16(np.clip(ref, -most, most), NP16[dtype])
    got = host16(k)
    assert np.array_equal(got, from16(lim, NP16[dtype]), equal_nan=True)
    assert np.isfinite(got[:6]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,group", SHAPES)
def test_step_shapes(c4, D, group, dtype):
    pr = Problem(c4, [(77, 1), (1, 1), (0, 1), (16, 1), (200, 1)], H=2, D=D, group=group, dtype=dtype).fill()
    q = cuda16(pr.rng.standard_normal((5, 8, D)).astype(np.float32), dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse)
    again = pr.cache.attend(q, c4.Batch4(torch.from_numpy(pr.table).cuda(), torch.from_numpy(pr.lens).cuda()))
    assert torch.equal(out, again)  # without start, and without lse: the same bits


@pytest.mark.parametrize("P", [16, 32, 48, 64, 128, 1024])
@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 5), (5, 1), (8, 1), (12, 4), (16, 1), (34, 2), (3, 1)])
def test_step_heads_and_pages(c4, P, Hq, H):
    pr = Problem(c4, [(130, 1), (1031, 1), (63, 1), (64, 1), (65, 1)], P=P, H=H, D=64, group=32, dtype=torch.bfloat16, seed=P + Hq).fill()
    q = cuda16(pr.rng.standard_normal((5, Hq, 64)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=40)


@pytest.mark.parametrize("window", [0, 1, 7, 64, 65, 300])
@pytest.mark.parametrize("rows", [1, 2, 5, 8, 9, 17])
def test_few_rows_and_windows(c4, rows, window):
    pr = Problem(c4, [(300, rows), (rows, rows), (40, min(rows, 3)), (0, 0), (129, 1)], H=2, D=128, dtype=torch.float16, seed=rows).fill()
    q = cuda16(pr.rng.standard_normal((int(pr.start[-1]), 8, 128)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), window=window, return_lse=True, scale=0.11)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, window=window, scale=0.11, sample=150)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,group,Hq,H", [(64, 32, 4, 4), (64, 64, 16, 2), (128, 32, 5, 1), (128, 64, 8, 2), (128, 128, 3, 1),
                                          (256, 64, 4, 2), (256, 128, 12, 1), (256, 32, 2, 1)])
def test_chunks(c4, D, group, Hq, H, dtype):
    """Prompts from nothing, behind a prefix, of odd lengths, beside single tokens."""
    pr = Problem(c4, [(257, 257), (700, 131), (33, 33), (450, 1), (640, 128)], P=64, H=H, D=D, group=group, dtype=dtype, seed=D + Hq).fill()
    q = cuda16(pr.rng.standard_normal((int(pr.start[-1]), Hq, D)).astype(np.float32), dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=200)


@pytest.mark.parametrize("window", [1, 100, 129, 512])
def test_chunks_with_a_window(c4, window):
    pr = Problem(c4, [(900, 300), (200, 200)], P=32, H=1, D=128, dtype=torch.bfloat16, seed=window).fill()
    q = cuda16(pr.rng.standard_normal((500, 4, 128)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), window=window, return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, window=window, sample=200)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype,qs,ks,vs", [(torch.float16, 1e-3, 1.0, 1e-5), (torch.float16, 300.0, 0.01, 2e4), (torch.float16, 1e-6, 3e3, 1.0),
                                            (torch.bfloat16, 1e6, 1e-6, 1e30), (torch.bfloat16, 1e-6, 1e6, 1e-30), (torch.bfloat16, 30.0, 0.1, 1e5)])
def test_magnitudes(c4, dtype, qs, ks, vs, rows):
    """Queries, keys and values far from one: no overflow, no loss of small ones."""
    pr = Problem(c4, [(150, rows), (60, rows)], H=1, D=128, dtype=dtype, seed=3)
    pr.k, pr.v = (from16(to16((x * f).astype(np.float32), pr.bf16), pr.bf16) for x, f in ((pr.k, ks), (pr.v, vs)))
    pr.fill()
    q = cuda16((pr.rng.standard_normal((2 * rows, 4, 128)) * qs).astype(np.float32), dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == (0 if np.isfinite(pr.k).all() and np.isfinite(pr.v).all() else 1)  # 2e4 reaches past binary16
    check_attention(pr, q, out, lse, sample=60)


@pytest.mark.parametrize("rows", [1, 3, 70])
def test_value_scales_differ_by_token(c4, rows):
    """Early tokens' values are tiny, later ones large, and the other way round."""
    pr = Problem(c4, [(500, rows), (400, rows)], H=1, D=128, dtype=torch.bfloat16, seed=8)
    pr.v[:, :250] *= 1e-4
    pr.v[:, 700:] *= 1e4
    pr.v = from16(to16(pr.v, True), True)
    pr.fill()
    q = cuda16(pr.rng.standard_normal((2 * rows, 4, 128)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    check_attention(pr, q, out, lse, sample=60)


@pytest.mark.parametrize("rows", [1, 2, 40])
def test_bad_batches_on_the_device(c4, rows):
    """Page ids outside the pool, lengths past the table, more rows than max_rows or
    than tokens: flagged, nothing outside is touched, the other sequences are served."""
    from kv_cache_compression_cg_gb300 import capi
    pr = Problem(c4, [(100, rows), (90, rows), (min(rows, 5), rows), (64, rows)], P=16, H=1, D=64, group=64, seed=rows)
    want = Problem(c4, [(100, rows), (90, rows), (min(rows, 5), rows), (64, rows)], P=16, H=1, D=64, group=64, seed=rows).fill()
    pr.fill()
    q = cuda16(pr.rng.standard_normal((4 * rows, 2, 64)).astype(np.float32), pr.dtype)
    good, glse = want.cache.attend(q, want.batch(), return_lse=True)
    assert want.flags() == 0
    empty = [int(pr.start[2]) + i for i in range(rows - min(rows, 5))]  # rows before their sequence's first token
    assert (good[empty] == 0).all() and torch.isneginf(glse[empty]).all()
    pr.table[1, 2] = pr.pages
    pr.table[3, 0] = -1
    before = pr.cache.pool.clone()
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == capi.CG_FLAG_BATCH
    r = rows
    assert torch.equal(out[:r], good[:r]) and torch.equal(out[2 * r:3 * r], good[2 * r:3 * r])
    check_attention(pr, q, out, lse, sample=60, hidden={(1, 2), (3, 0)})
    pr.cache.status.zero_()
    b = pr.batch([90 if n == 90 else r for n, r in pr.seqs])
    k, v = pr.cache.read(b)
    at = int(pr.start[1]) + 32
    assert pr.flags() == capi.CG_FLAG_BATCH
    assert (k[at:at + 16] == 0).all() and (v[at:at + 16] == 0).all() and (k[at - 1] != 0).any() and (k[at + 16] != 0).any()
    pr.cache.status.zero_()
    pr.cache.write(k, v, b)
    assert pr.flags() == capi.CG_FLAG_BATCH
    spare = np.setdiff1d(np.arange(pr.pages), pr.table)
    assert torch.equal(pr.cache.pool[0, spare], before[0, spare])
    # a length that the table cannot hold: what it holds is attended to
    pr.cache.status.zero_()
    lens = torch.tensor([pr.table.shape[1] * 16 + 1000, -5, 3, 2], dtype=torch.int32).cuda()
    pr.cache.attend(q, c4.Batch4(torch.zeros(4, 3, dtype=torch.int32).cuda(), lens, torch.from_numpy(pr.start).cuda(), rows=4 * rows, max_rows=rows))
    assert pr.flags() == capi.CG_FLAG_BATCH
    if rows > 1:  # the second sequence has more rows than the batch says: left out
        pr.cache.status.zero_()
        start = torch.tensor([0, 1, 1 + rows, 1 + rows, 1 + rows], dtype=torch.int32).cuda()
        o = torch.full_like(q, 5.0)
        pr.cache.attend(q, c4.Batch4(torch.from_numpy(want.table).cuda(), torch.from_numpy(pr.lens).cuda(), start, rows=4 * rows, max_rows=rows - 1), out=o)
        assert pr.flags() == capi.CG_FLAG_BATCH
        assert (o[1:] == 5.0).all() and (o[0] != 5.0).any()


@pytest.mark.parametrize("rows", [1, 50])
def test_masked_garbage_and_nan_keys(c4, rows):
    """A NaN in a key a row may see makes that row NaN, and no other row; a NaN behind a row's position does nothing."""
    pr = Problem(c4, [(100, rows), (100, rows)], H=1, D=128, seed=5)
    pr.k[0, 99, 0, 3] = np.nan       # last token of the first sequence
    pr.fill()
    assert pr.flags() == 1
    q = cuda16(pr.rng.standard_normal((2 * rows, 4, 128)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(out[rows - 1]).all()
    keep = [i for i in range(2 * rows) if i != rows - 1]
    assert torch.isfinite(out[keep]).all() and torch.isfinite(lse[keep]).all()


@pytest.mark.parametrize("rows", [1, 6, 50, 200])
@pytest.mark.parametrize("group", [32, 128])
def test_nan_values(c4, rows, group):
    """A NaN or an infinity in a value makes its group's channels NaN in the rows that see the token, and
    nothing else: not in rows before it, whose weight for it is none."""
    pr = Problem(c4, [(300, rows), (260, rows)], H=1, D=128, group=group, dtype=torch.bfloat16, seed=6)
    pr.v[0, 299 - rows // 2, 0, 3] = np.nan
    pr.v[0, 299 - rows // 3, 0, 70] = np.inf
    pr.v[0, 300 + 20, 0, 127] = -np.inf
    pr.fill()
    assert pr.flags() == 1
    q = cuda16(pr.rng.standard_normal((2 * rows, 3, 128)).astype(np.float32), pr.dtype)
    for window in (0, 40):
        out, lse = pr.cache.attend(q, pr.batch(), window=window, return_lse=True)
        check_attention(pr, q, out, lse, window=window, sample=150)


@pytest.mark.parametrize("rows", [1, 33])
def test_same_bits_every_time_and_on_another_stream(c4, rows):
    pr = Problem(c4, [(3000, rows), (77, rows), (1500, rows)], P=64, H=2, D=128, dtype=torch.bfloat16).fill()
    q = cuda16(pr.rng.standard_normal((3 * rows, 8, 128)).astype(np.float32), pr.dtype)
    b = pr.batch()
    first = pr.cache.attend(q, b, return_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for i in range(6):
        outs.append(pr.cache.attend(q, b, return_lse=True, stream=side if i % 2 else None))
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])


@pytest.mark.parametrize("rows", [1, 48])
def test_step_in_a_graph(c4, rows):
    """Write and attend captured once and replayed with longer sequences."""
    pr = Problem(c4, [(900, rows), (500, rows)], P=32, H=2, D=64, group=64, dtype=torch.float16).fill()
    ref = Problem(c4, [(900, rows), (500, rows)], P=32, H=2, D=64, group=64, dtype=torch.float16).fill()
    b = pr.batch()
    kv = [cuda16(np.concatenate([x[0][pr.token(s, n - r):pr.token(s, n - r) + r] for s, (n, r) in enumerate(pr.seqs)]), pr.dtype) for x in (pr.k, pr.v)]
    q = cuda16(pr.rng.standard_normal((2 * rows, 4, 64)).astype(np.float32), pr.dtype)
    out = torch.empty_like(q)
    b.kv_len.copy_(torch.tensor([400, 300], dtype=torch.int32))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            pr.cache.write(*kv, b)
            pr.cache.attend(q, b, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pr.cache.write(*kv, b)
        pr.cache.attend(q, b, out=out)
    pr.fill()
    b.kv_len.copy_(torch.from_numpy(pr.lens))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.cache.attend(q, ref.batch())
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_offsets_past_32_bits(c4):
    """Pages beyond the pool's first 4 GB, of a later layer."""
    pages = 30000
    pool = torch.empty(2 * pages * 8 * 4 * 2304, dtype=torch.uint8, device="cuda")
    cache = c4.Cache4(2, pages, 64, 8, 128, pool=pool)
    assert cache.nbytes > 2 ** 32
    rng = np.random.default_rng(0)
    ids = torch.tensor([[pages - 1, pages - 7, 5]], dtype=torch.int32).cuda()
    b = c4.Batch4(ids, torch.tensor([150], dtype=torch.int32).cuda(), torch.tensor([0, 150], dtype=torch.int32).cuda(), rows=150)
    x = rng.standard_normal((2, 150, 8, 128)).astype(np.float32)
    k, v = (cuda16(y, torch.float16) for y in x)
    small = c4.Cache4(1, 3, 64, 8, 128)
    sb = c4.Batch4(torch.arange(3, dtype=torch.int32).cuda().reshape(1, 3), b.kv_len, b.start, rows=150)
    cache.write(k, v, b, layer=1)
    small.write(k, v, sb)
    q = cuda16(rng.standard_normal((150, 16, 128)).astype(np.float32), torch.float16)
    for x, y in zip(cache.read(b, layer=1), small.read(sb)):
        assert torch.equal(x, y)
    assert torch.equal(cache.attend(q, b, layer=1), small.attend(q, sb))
    one = c4.Batch4(ids, b.kv_len)
    assert torch.equal(cache.attend(q[:1], one, layer=1), small.attend(q[:1], c4.Batch4(sb.table, b.kv_len)))
    assert int(cache.status.item()) == 0


def test_wrapper_refusals(c4):
    cache = c4.Cache4(2, 4, 16, 2, 64)
    i = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    b = c4.Batch4(i, i[:, 0].contiguous())
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        c4.Batch4(i, i[:, 0])
    with pytest.raises(ValueError):
        c4.Batch4(i, i[:2, 0].contiguous())
    with pytest.raises(ValueError, match="rows"):
        c4.Batch4(i, i[:, 0].contiguous(), torch.zeros(4, dtype=torch.int32, device="cuda"))
    for bad in (x.float(), x.bfloat16()):
        with pytest.raises(TypeError):
            cache.write(bad, x, b)
    for bad in (x[:2], x.transpose(0, 1), x.cpu(), x[:, :, :32]):
        with pytest.raises(ValueError):
            cache.write(x, bad, b)
    with pytest.raises(Exception):
        cache.write(x, x, b, layer=2)
    with pytest.raises(TypeError):
        cache.read(b, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cache.read(b, out=(x, x[:2]))
    with pytest.raises(TypeError):
        cache.attend(q.float(), b)
    for bad in (q[:, :3], q[:2], q[..., :32], q[:, :0]):
        with pytest.raises(ValueError):
            cache.attend(bad, b)
    with pytest.raises(ValueError):
        cache.attend(q, b, out=torch.empty(3, 4, 64, dtype=torch.float32, device="cuda"))
    with pytest.raises(ValueError):
        c4.Cache4(2, 4, 16, 2, 64, pool=cache.pool[:1])
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("rows", [1, 5, 40])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_that_are_not_positive(c4, rows, scale):
    """Equal weights (scale 0) and reversed ones."""
    pr = Problem(c4, [(150, rows), (60, rows)], H=1, D=128, dtype=torch.float16, seed=4).fill()
    q = cuda16(pr.rng.standard_normal((2 * rows, 4, 128)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True, scale=scale)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, scale=scale, sample=60)


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("B", [33, 700, 1500])
def test_many_sequences(c4, B, rows):
    """More sequences than one look at the batch takes, some without rows, lengths from none to a few pages."""
    rng = np.random.default_rng(B)
    seqs = [(int(n), int(min(r, n)) if n else 0) for n, r in zip(rng.integers(0, 70, B), rng.integers(0, rows + 1, B))]
    seqs[0], seqs[-1] = (0, 0), (40, rows)
    pr = Problem(c4, seqs, P=16, H=1, D=64, group=64, seed=B).fill()
    q = cuda16(pr.rng.standard_normal((int(pr.start[-1]), 4, 64)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=300)


def test_many_chunks(c4):
    """The same with chunks: pairs of row tiles over many sequences, long ones between."""
    rng = np.random.default_rng(7)
    seqs = [(int(n), int(r)) for n, r in zip(rng.integers(60, 90, 40), rng.integers(20, 60, 40))]
    seqs[11], seqs[12], seqs[35] = (900, 700), (0, 0), (1400, 260)
    pr = Problem(c4, seqs, P=48, H=2, D=64, group=32, dtype=torch.bfloat16).fill()
    q = cuda16(pr.rng.standard_normal((int(pr.start[-1]), 8, 64)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=300)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 128)])
def test_steps_beside_a_chunk(c4, D, group):
    """One prompt among many single tokens: either kernel on its own sequences."""
    seqs = [(200 + i, 1) for i in range(30)] + [(500, 77)] + [(3, 3), (90, 2)]
    pr = Problem(c4, seqs, P=32, H=1, D=D, group=group, dtype=torch.bfloat16).fill()
    q = cuda16(pr.rng.standard_normal((int(pr.start[-1]), 4, D)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=250)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
@pytest.mark.parametrize("rows", [1, 60, 300])
def test_one_head_over_a_long_context(c4, D, group, rows):
    """One KV head: its keys are split over the whole GPU and joined."""
    pr = Problem(c4, [(12345, rows)], P=64, H=1, D=D, group=group, dtype=torch.float16).fill()
    q = cuda16(pr.rng.standard_normal((rows, 2, D)).astype(np.float32), pr.dtype)
    out, lse = pr.cache.attend(q, pr.batch(), return_lse=True)
    assert pr.flags() == 0
    check_attention(pr, q, out, lse, sample=24)
    for _ in range(3):
        again = pr.cache.attend(q, pr.batch(), return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("pad", [4, 3])
def test_strided_queries_and_outputs(c4, rows, pad):
    """Queries sliced out of wider rows, outputs into wider ones; rows that no sequence has stay as they are."""
    pr = Problem(c4, [(90, rows), (50, rows)], H=2, D=64, group=32, dtype=torch.bfloat16).fill()
    n = 2 * rows
    wide = torch.zeros(n + 2, 4 * 64 + pad, dtype=pr.dtype, device="cuda")
    q = wide[:, pad:].unflatten(1, (4, 64))
    q.copy_(cuda16(pr.rng.standard_normal((n + 2, 4, 64)).astype(np.float32), pr.dtype))
    into = torch.full((n + 2, 4 * 64 + pad), 9.0, dtype=pr.dtype, device="cuda")
    out = into[:, pad:].unflatten(1, (4, 64))
    b = c4.Batch4(torch.from_numpy(pr.table).cuda(), torch.from_numpy(pr.lens).cuda(), torch.from_numpy(pr.start).cuda(), rows=n + 2, max_rows=rows)
    pr.cache.attend(q, b, out=out)
    assert pr.flags() == 0
    check_attention(pr, q[:n].contiguous(), out[:n].contiguous(), None, sample=100)
    assert (into[:, :pad] == 9.0).all() and (into[n:] == 9.0).all()
    plain = pr.cache.attend(q[:n].contiguous(), pr.batch())
    assert torch.equal(plain, out[:n])


def test_example_serves_from_a_restored_prefix(c4):
    """compress -> restore -> write into the cache -> decode in a graph. The attention's error against plain attention
    over the cache's own values: one rounding each of weights, values and output to binary16 (2^-11), all against the
    weighted mean of |v|, and the scores' and exponentials' 2^-15 (scores up to 30, 8 u each and 2^-19)."""
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_from_prefix.py")
    spec = importlib.util.spec_from_file_location("serve_from_prefix", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off = m.serve(layers=2, tokens=300, steps=3, say=lambda *a: None)
    assert 0.0 < off <= 3 * 2.0 ** -11 + 2.0 ** -15
