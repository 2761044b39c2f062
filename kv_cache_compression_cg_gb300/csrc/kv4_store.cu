// kv4_store.cu - writing rows into the 4-bit paged cache (Z) and reading them
// back (U); include/cachegen.h has the formulas and the record layout.
//
// A warp owns 8 consecutive rows of the batch, one KV head and one layer, K and V.
// Every row finds its own slot, so rows of several sequences, ends of pages and
// odd positions need no cases of their own: a token's bytes are its own, no byte
// is shared between two tokens, and nothing is read before it is written.
//   K: lane (row g = lane / 4, chunk t = lane % 4) holds channels 16j + 4t + 0..3,
//      j = 0 .. D/16 - 1: the four lanes of a row read whole 32-byte sectors and
//      each stores its chunk of D/8 bytes. A group's range is taken in the lane's
//      registers, then over the four lanes.
//   V: lane (row r = lane / 8, piece g = lane % 8), two rows a lane, holds channels
//      g*D/8 + 0 .. D/8 - 1; a group's range goes over the pieces that share it.
// Bound by HBM: 4 bytes a K, V pair of values on the 16-bit side, 1 + 1/(group/8)
// stored.
#include "kv4.cuh"

namespace cg {
namespace {

// s of Z from a group's range: NaN where the range is not finite.
template <bool BF>
__device__ __forceinline__ float group_scale(float lo, float hi) {
    const float range = __fsub_rn(hi, lo);
    if (!(fabsf(range) <= 3.402823466e38f)) return __uint_as_float(0x7FC00000u);
    const unsigned b = (__float_as_uint(__fdiv_rn(range, 15.0f)) + 0x10000u) & ~0x1FFFFu;  // seven significant bits
    return bits_to_float<BF>(float_to_bits<BF>(__uint_as_float(b)));
}

__device__ __forceinline__ unsigned code_of(float x, float lo, float s) {
    if (!(s > 0.0f)) return 0u;
    return (unsigned)__float2int_rn(fminf(__fdiv_rn(__fsub_rn(x, lo), s), 15.0f));
}

// Two 16-bit values side by side: the lesser, the greater of each, NaNs kept.
template <bool BF>
__device__ __forceinline__ unsigned min_pair(unsigned a, unsigned b) {
    unsigned y;
    if (BF) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
template <bool BF>
__device__ __forceinline__ unsigned max_pair(unsigned a, unsigned b) {
    unsigned y;
    if (BF) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// The range of a group: N pairs of this lane, and those of the lanes `from`, 2 from, ... `to` / 2 away.
template <bool BF, int N>
__device__ __forceinline__ void range_of(const unsigned *x, int from, int to, float &lo, float &hi) {
    unsigned a = x[0], b = x[0];
#pragma unroll
    for (int i = 1; i < N; i++) {
        a = min_pair<BF>(a, x[i]);
        b = max_pair<BF>(b, x[i]);
    }
#pragma unroll
    for (int o = from; o < to; o <<= 1) {
        a = min_pair<BF>(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        b = max_pair<BF>(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    }
    a = min_pair<BF>(a, a >> 16);
    b = max_pair<BF>(b, b >> 16);
    lo = bits_to_float<BF>(a & 0xFFFFu);
    hi = bits_to_float<BF>(b & 0xFFFFu);
}

// The codes of N pairs of one group into words: pair j's go to nibbles nib(j), nib2(j) of word j / 4.
// rint((x - lo) / s) without a division: y = (x - lo) (1/s) is within 2^-19 of the quotient, so its nearest
// whole number is the quotient's unless y lies that close to halfway; then (or where s is none, or so small
// that its own rounding let the quotient pass 15) the eight values of the word are divided.
template <bool BF, int N, typename Nib, typename Nib2>
__device__ __forceinline__ void codes_of(const unsigned *x, float lo, float hi, float s, unsigned *words, Nib nib,
                                         Nib2 nib2) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: y + kMagic has y's nearest whole number in its last bits
    const bool plain = s > 1e-30f && hi - lo <= 15.4f * s;  // 1/s far from its own limits
    const float r = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int i = 0; i < N / 4; i++) {
        unsigned w = 0, sub = 0;
        float far = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const unsigned pair = x[4 * i + j / 2];
            const int at = 4 * (j & 1 ? nib2(j / 2) : nib(j / 2));
            const float d = __fsub_rn(bits_to_float<BF>(j & 1 ? pair >> 16 : pair & 0xFFFFu), lo);
            const float n = __fmaf_rn(d, r, kMagic);
            far = fmaxf(far, fabsf(__fmaf_rn(d, r, __fsub_rn(kMagic, n))));
            w += __float_as_uint(n) << at;
            sub += 0x4B400000u << at;
        }
        w -= sub;
        if (!(plain && far <= 0.49999f)) {
            w = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const unsigned pair = x[4 * i + j / 2];
                w |= code_of(bits_to_float<BF>(j & 1 ? pair >> 16 : pair & 0xFFFFu), lo, s)
                     << (4 * (j & 1 ? nib2(j / 2) : nib(j / 2)));
            }
        }
        words[i] = w;
    }
}

// N pairs from p; VEC: p is aligned for loads of 8 bytes (N = 2) or 16.
template <int N, bool VEC>
__device__ __forceinline__ void load_pairs(const uint16_t *p, unsigned *x) {
    if (VEC && N == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
        x[0] = w.x;
        x[1] = w.y;
    } else if (VEC) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
            x[i] = w.x;
            x[i + 1] = w.y;
            x[i + 2] = w.z;
            x[i + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) x[i] = __ldg(p + 2 * i) | ((unsigned)__ldg(p + 2 * i + 1) << 16);
    }
}

template <int W>
__device__ __forceinline__ void store_words(uint8_t *p, const unsigned *w) {
    if (W == 1) {
        *reinterpret_cast<unsigned *>(p) = w[0];
    } else if (W == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4)
            *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *p, unsigned *w) {
    if (W == 1) {
        w[0] = *reinterpret_cast<const unsigned *>(p);
    } else if (W == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x;
        w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = u.x;
            w[i + 1] = u.y;
            w[i + 2] = u.z;
            w[i + 3] = u.w;
        }
    }
}

// The warp's unit of work: head fastest, so that the warps of a CTA read
// neighbouring heads of the same rows.
struct Unit {
    int tile, head, layer;
};
__device__ __forceinline__ Unit unit_of(const Kv4 &p, long long w, int tiles) {
    Unit u;
    u.head = (int)(w % p.H);
    w /= p.H;
    u.tile = (int)(w % tiles);
    u.layer = (int)(w / tiles);
    return u;
}

// Record of row r's slot, head h, in layer l of the pool: nullptr where it has
// none. tok = its place in the record.
__device__ __forceinline__ long long slot_of(const Kv4 &p, int r, int h, int l, int &tok, bool &mine, int32_t *status) {
    int b;
    long long pos;
    mine = r < p.rows && row_pos(p, r, b, pos, status);
    if (!mine) return -1;
    const int page = page_of(p, b, pos, status);
    if (page < 0) return -1;
    const int at = (int)(pos % p.P);
    tok = at % kBlk;
    return l * p.layer_stride + page * p.page_stride + ((long long)h * (p.P / kBlk) + at / kBlk) * p.record;
}

template <int D, int G, bool BF, bool VEC>
__global__ void __launch_bounds__(256) k_kv4_write(uint8_t *__restrict__ pool, Kv4 p, int layer, int nlayers, int tiles,
                                                   const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
                                                   long long krs, long long vrs, long long kls, long long vls,
                                                   int32_t *status) {
    using R = Rec<D, G>;
    constexpr int W = D / 32;              // words of a K chunk
    constexpr int N = D / 8;               // channels of a V piece
    constexpr int GP = G / N;              // pieces a group
    static_assert(G >= N, "a piece lies in one group");
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (w >= (long long)tiles * p.H * nlayers) return;
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane & 7;
    const Unit u = unit_of(p, w, tiles);
    // rows past the end load the last one's values and store nothing: no load waits for the slots
    const int last = p.rows - 1, row = u.tile * 8 + (lane >> 2);
    unsigned x[D / 8], z[2][N / 2];  // pairs
    const uint16_t *src = k + u.layer * kls + min(row, last) * krs + (long long)u.head * D + 4 * t;
#pragma unroll
    for (int j = 0; j < D / 16; j++) load_pairs<2, VEC>(src + 16 * j, x + 2 * j);
#pragma unroll
    for (int half = 0; half < 2; half++) {
        src = v + u.layer * vls + min(u.tile * 8 + half * 4 + (lane >> 3), last) * vrs + (long long)u.head * D + g * N;
        load_pairs<N / 2, VEC>(src, z[half]);
    }
    int tok = 0;
    bool mine, bad = false;
    const long long at = slot_of(p, row, u.head, layer + u.layer, tok, mine, status);
    {
        unsigned words[W], params[R::NG];
#pragma unroll
        for (int i = 0; i < R::NG; i++) {
            const unsigned *y = x + i * (G / 8);
            float lo, hi;
            range_of<BF, G / 8>(y, 1, 4, lo, hi);
            const float s = group_scale<BF>(lo, hi);
            // pair j of a word: channels e = 0, 1 (even j) or 2, 3 of step 2w + j / 2
            codes_of<BF, G / 8>(y, lo, hi, s, words + i * (G / 32), [](int j) { return 2 * (j >> 1) + (j & 1); },
                                [](int j) { return 4 + 2 * (j >> 1) + (j & 1); });
            if (s != s) {
                bad |= at >= 0;
                lo = s;
            }
            params[i] = float_to_bits<BF>(s) | (float_to_bits<BF>(lo) << 16);
        }
        if (at >= 0) {
            uint8_t *rec = pool + at;
            store_words<W>(rec + (tok >> 3) * (4 * D) + (tok & 7) * (D / 2) + t * (D / 8), words);
#pragma unroll
            for (int i = 0; i < R::NG; i++)
                if ((i & 3) == t) *reinterpret_cast<unsigned *>(rec + R::kPK + (tok * R::NG + i) * 4) = params[i];
        }
    }
#pragma unroll
    for (int half = 0; half < 2; half++) {
        const int from = (half * 4 + (lane >> 3)) * 4;  // the lane that looked this row's slot up
        const long long vat = __shfl_sync(0xFFFFFFFFu, at, from);
        const int vtok = __shfl_sync(0xFFFFFFFFu, tok, from);
        float lo, hi;
        range_of<BF, N / 2>(z[half], 1, GP, lo, hi);
        const float s = group_scale<BF>(lo, hi);
        unsigned words[N / 8];
        codes_of<BF, N / 2>(z[half], lo, hi, s, words, [](int j) { return 2 * j; }, [](int j) { return 2 * j + 1; });
        if (s != s) {
            bad |= vat >= 0;
            lo = s;
        }
        if (vat >= 0) {
            uint8_t *rec = pool + vat;
            store_words<N / 8>(rec + R::kV + (vtok >> 3) * (4 * D) + g * (D / 2) + (vtok & 7) * (D / 16), words);
            if (g % GP == 0)
                *reinterpret_cast<unsigned *>(rec + R::kPV + (vtok * R::NG + g / GP) * 4) =
                    float_to_bits<BF>(s) | (float_to_bits<BF>(lo) << 16);
        }
    }
    if (bad) raise_flag(status, CG_FLAG_NONFINITE);
}

// 8 (or 4) values to p in the output type; values past binary16's (bfloat16's)
// largest become it.
template <int OUT>  // 0: binary32, 1: binary16, 2: bfloat16
__device__ __forceinline__ unsigned half_bits(float x) {
    const float most = OUT == 1 ? 65504.0f : 3.3895313892515355e38f;
    if (x > most) x = most;  // NaN stays
    if (x < -most) x = -most;
    return float_to_bits<OUT == 2>(x);
}
template <int OUT, bool VEC, int N>
__device__ __forceinline__ void store_values(void *base, long long at, const float *x) {
    if (OUT == 0) {
        float *p = static_cast<float *>(base) + at;
        if (VEC) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) p[i] = x[i];
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        if (VEC) {
            unsigned w[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; i++) w[i] = half_bits<OUT>(x[2 * i]) | (half_bits<OUT>(x[2 * i + 1]) << 16);
            store_words<N / 2>(reinterpret_cast<uint8_t *>(p), w);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) p[i] = (uint16_t)half_bits<OUT>(x[i]);
        }
    }
}

__device__ __forceinline__ float code_value(unsigned word, int nib, float s, float lo) {
    // 2^23 + c as bits, less 2^23: no conversion instruction; the product is exact, so one rounding
    const float c = __uint_as_float(((word >> (4 * nib)) & 15u) | 0x4B000000u) - 8388608.0f;
    return __fmaf_rn(c, s, lo);
}

template <int D, int G, int OUT, bool BF, bool VEC>
__global__ void __launch_bounds__(256) k_kv4_read(const uint8_t *__restrict__ pool, Kv4 p, int layer, int nlayers,
                                                  int tiles, void *ok, void *ov, long long rs, long long ls,
                                                  int32_t *status) {
    using R = Rec<D, G>;
    constexpr int W = D / 32;
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (w >= (long long)tiles * p.H * nlayers) return;
    const int lane = threadIdx.x & 31;
    const Unit u = unit_of(p, w, tiles);
    const int row = u.tile * 8 + (lane >> 2), t = lane & 3, g = lane & 7;
    int tok = 0;
    bool mine;
    const long long at = slot_of(p, row, u.head, layer + u.layer, tok, mine, status);
    constexpr int N = D / 8;
    unsigned words[W], params[R::NG], vw[2][N / 8], vp[2];
#pragma unroll
    for (int i = 0; i < W; i++) words[i] = 0;
#pragma unroll
    for (int i = 0; i < R::NG; i++) params[i] = 0;
    if (at >= 0) {
        const uint8_t *rec = pool + at;
        load_words<W>(rec + (tok >> 3) * (4 * D) + (tok & 7) * (D / 2) + t * (D / 8), words);
#pragma unroll
        for (int i = 0; i < R::NG; i++)
            params[i] = *reinterpret_cast<const unsigned *>(rec + R::kPK + (tok * R::NG + i) * 4);
    }
    bool vmine[2];
#pragma unroll
    for (int half = 0; half < 2; half++) {
        const int from = (half * 4 + (lane >> 3)) * 4;  // the lane that looked this row's slot up
        const long long vat = __shfl_sync(0xFFFFFFFFu, at, from);
        const int vtok = __shfl_sync(0xFFFFFFFFu, tok, from);
        vmine[half] = __shfl_sync(0xFFFFFFFFu, (int)mine, from);
        vp[half] = 0;
#pragma unroll
        for (int i = 0; i < N / 8; i++) vw[half][i] = 0;
        if (vat >= 0) {
            const uint8_t *rec = pool + vat;
            load_words<N / 8>(rec + R::kV + (vtok >> 3) * (4 * D) + g * (D / 2) + (vtok & 7) * (D / 16), vw[half]);
            vp[half] = *reinterpret_cast<const unsigned *>(rec + R::kPV + (vtok * R::NG + g * N / G) * 4);
        }
    }
    if (mine) {
        const long long dst = u.layer * ls + row * rs + (long long)u.head * D + 4 * t;
#pragma unroll
        for (int j = 0; j < D / 16; j++) {
            const unsigned pr = params[16 * j / G];
            const float s = bits_to_float<BF>(pr & 0xFFFFu), lo = bits_to_float<BF>(pr >> 16);
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = code_value(words[j >> 1], 4 * (e & 1) + 2 * (j & 1) + (e >> 1), s, lo);
            store_values<OUT, VEC, 4>(ok, dst + 16 * j, x);
        }
    }
#pragma unroll
    for (int half = 0; half < 2; half++) {
        if (!vmine[half]) continue;
        const float s = bits_to_float<BF>(vp[half] & 0xFFFFu), lo = bits_to_float<BF>(vp[half] >> 16);
        const long long dst = u.layer * ls + (u.tile * 8 + half * 4 + (lane >> 3)) * rs + (long long)u.head * D + g * N;
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = code_value(vw[half][i / 8], j, s, lo);
            store_values<OUT, VEC, 8>(ov, dst + i, x);
        }
    }
}

bool multiple(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <int D, int G>
cudaError_t write_dg(uint8_t *pool, const Kv4 &p, int layer, int nl, const void *kv, const void *vv, long long krs,
                     long long vrs, long long kls, long long vls, int32_t *status, cudaStream_t s) {
    const uint16_t *k = static_cast<const uint16_t *>(kv), *v = static_cast<const uint16_t *>(vv);
    const int tiles = (p.rows + 7) / 8;
    const unsigned blocks = (unsigned)(((long long)tiles * p.H * nl + 7) / 8);
    const bool vec = multiple(k, 16) && multiple(v, 16) && krs % 8 == 0 && vrs % 8 == 0 && kls % 8 == 0 && vls % 8 == 0;
#define CG_KV4_GO(BF, VEC) \
    k_kv4_write<D, G, BF, VEC><<<blocks, 256, 0, s>>>(pool, p, layer, nl, tiles, k, v, krs, vrs, kls, vls, status)
    if (p.dtype == CG_DT_BF16) vec ? CG_KV4_GO(true, true) : CG_KV4_GO(true, false);
    else vec ? CG_KV4_GO(false, true) : CG_KV4_GO(false, false);
#undef CG_KV4_GO
    return cudaGetLastError();
}

template <int D, int G>
cudaError_t read_dg(const uint8_t *pool, const Kv4 &p, int layer, int nl, bool f32, void *ok, void *ov, long long rs,
                    long long ls, int32_t *status, cudaStream_t s) {
    const int tiles = (p.rows + 7) / 8;
    const unsigned blocks = (unsigned)(((long long)tiles * p.H * nl + 7) / 8);
    const bool vec = multiple(ok, 16) && multiple(ov, 16) && rs % (f32 ? 4 : 8) == 0 && ls % (f32 ? 4 : 8) == 0;
    const bool bf = p.dtype == CG_DT_BF16;
#define CG_KV4_GO(OUT, BF, VEC) \
    k_kv4_read<D, G, OUT, BF, VEC><<<blocks, 256, 0, s>>>(pool, p, layer, nl, tiles, ok, ov, rs, ls, status)
    if (f32) {
        if (bf) vec ? CG_KV4_GO(0, true, true) : CG_KV4_GO(0, true, false);
        else vec ? CG_KV4_GO(0, false, true) : CG_KV4_GO(0, false, false);
    } else if (bf) {
        vec ? CG_KV4_GO(2, true, true) : CG_KV4_GO(2, true, false);
    } else {
        vec ? CG_KV4_GO(1, false, true) : CG_KV4_GO(1, false, false);
    }
#undef CG_KV4_GO
    return cudaGetLastError();
}

}  // namespace

#define CG_KV4_SHAPES(CALL)                                  \
    switch (p.D * 1000 + p.G) {                              \
        case 64032: return CALL(64, 32);                     \
        case 64064: return CALL(64, 64);                     \
        case 128032: return CALL(128, 32);                   \
        case 128064: return CALL(128, 64);                   \
        case 128128: return CALL(128, 128);                  \
        case 256032: return CALL(256, 32);                   \
        case 256064: return CALL(256, 64);                   \
        case 256128: return CALL(256, 128);                  \
        default: return cudaErrorInvalidValue;               \
    }

cudaError_t launch_kv4_write(uint8_t *pool, const Kv4 &p, int layer, int nl, const void *k, const void *v,
                             long long krs, long long vrs, long long kls, long long vls, int32_t *status,
                             cudaStream_t s) {
#define CALL(D, G) write_dg<D, G>(pool, p, layer, nl, k, v, krs, vrs, kls, vls, status, s)
    CG_KV4_SHAPES(CALL)
#undef CALL
}

cudaError_t launch_kv4_read(const uint8_t *pool, const Kv4 &p, int layer, int nl, bool f32, void *ok, void *ov,
                            long long rs, long long ls, int32_t *status, cudaStream_t s) {
#define CALL(D, G) read_dg<D, G>(pool, p, layer, nl, f32, ok, ov, rs, ls, status, s)
    CG_KV4_SHAPES(CALL)
#undef CALL
}

}  // namespace cg
