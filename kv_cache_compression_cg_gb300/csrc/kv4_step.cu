// kv4_step.cu - attention over the 4-bit paged cache (N in include/cachegen.h).
//
// One CTA a (row, query head); its warps take every fourth key, the lanes the
// channels; an online softmax a warp, joined through shared memory at the end.
#include "kv4.cuh"

namespace cg {
namespace {

template <int D, int G, bool BF>
__global__ void __launch_bounds__(128) k_kv4_rows(Kv4 p, Kv4Attend a) {
    using R = Rec<D, G>;
    constexpr int N = D / 32;  // channels a lane: lane + 32 i
    __shared__ float sm[4], sl[4], so[4][D];
    const int row = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, kvh = h / a.R;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int b;
    long long pos;
    if (!row_pos(p, row, b, pos, a.status)) return;
    const int len = seq_len(p, b, a.status);
    const long long last = pos < len ? pos : (long long)len - 1;
    const long long first = a.window && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    float q[N], o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        q[i] = bits_to_float<BF>(a.q[row * a.q_stride + (long long)h * D + lane + 32 * i]) * a.scale;
        o[i] = 0.0f;
    }
    for (long long j = first + warp; j <= last; j += 4) {
        const int page = page_of(p, b, j, a.status);
        if (page < 0) continue;
        const int at = (int)(j % p.P), tok = at % kBlk;
        const uint8_t *rec = a.pool + page * p.page_stride + ((long long)kvh * (p.P / kBlk) + at / kBlk) * p.record;
        float s = 0.0f, vv[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int d = lane + 32 * i, w = d / 32, e = d % 16;
            const int nib = 4 * (e & 1) + 2 * (d / 16 % 2) + ((e >> 1) & 1);
            const unsigned kb = rec[tok * (D / 2) + (e / 4) * (D / 8) + w * 4 + nib / 2];
            const unsigned kp = *reinterpret_cast<const unsigned *>(rec + R::kPK + (tok * R::NG + d / G) * 4);
            s += q[i] * fmaf((float)((kb >> (4 * (nib & 1))) & 15u), bits_to_float<BF>(kp & 0xFFFFu),
                             bits_to_float<BF>(kp >> 16));
            const int g = d / (D / 8), c = d % (D / 8);
            const unsigned vb = rec[R::kV + (tok >> 3) * (4 * D) + g * (D / 2) + (tok & 7) * (D / 16) + c / 2];
            const unsigned vp = *reinterpret_cast<const unsigned *>(rec + R::kPV + (tok * R::NG + d / G) * 4);
            vv[i] = fmaf((float)((vb >> (4 * (c & 1))) & 15u), bits_to_float<BF>(vp & 0xFFFFu),
                         bits_to_float<BF>(vp >> 16));
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float top = fmaxf(m, s), f = expf(m - top), e = expf(s - top);
        m = top;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < N; i++) o[i] = o[i] * f + e * vv[i];
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < N; i++) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = sm[0], total = 0.0f;
    for (int w = 1; w < 4; w++) top = fmaxf(top, sm[w]);
    float f[4];
    for (int w = 0; w < 4; w++) {
        f[w] = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - top);
        total += sl[w] * f[w];
    }
    for (int d = threadIdx.x; d < D; d += 128) {
        float x = 0.0f;
        for (int w = 0; w < 4; w++) x += so[w][d] * f[w];
        a.out[row * a.out_stride + (long long)h * D + d] =
            (uint16_t)float_to_bits<BF>(top == -INFINITY ? 0.0f : x / total);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(long long)row * a.Hq + h] = top == -INFINITY ? top : top + logf(total);
}

template <int D, int G>
cudaError_t step_dg(const Kv4 &p, const Kv4Attend &a, cudaStream_t s) {
    const long long n = (long long)p.rows * a.Hq;
    if (p.dtype == CG_DT_BF16) k_kv4_rows<D, G, true><<<(unsigned)n, 128, 0, s>>>(p, a);
    else k_kv4_rows<D, G, false><<<(unsigned)n, 128, 0, s>>>(p, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_step(const Kv4 &p, const Kv4Attend &a, cudaStream_t s) {
    switch (p.D * 1000 + p.G) {
        case 64032: return step_dg<64, 32>(p, a, s);
        case 64064: return step_dg<64, 64>(p, a, s);
        case 128032: return step_dg<128, 32>(p, a, s);
        case 128064: return step_dg<128, 64>(p, a, s);
        case 128128: return step_dg<128, 128>(p, a, s);
        case 256032: return step_dg<256, 32>(p, a, s);
        case 256064: return step_dg<256, 64>(p, a, s);
        case 256128: return step_dg<256, 128>(p, a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace cg
