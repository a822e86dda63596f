// latent_rows.cu -- writing and reading back the latent cache: latent_append (RMSNorm of the latent
// part, rotary embedding of the rest, quantise on write at (sequence, position)) and latent_gather
// (rows of ragged runs of positions, dequantised, packed for the expanded form's projection).
//
// Both are HBM-bound: append reads 2c bytes (bf16) and writes R + 2 rd + 4 a row, gather the other
// way round.  A warp takes a row at a time: a lane holds 8 (append) or 16 (gather) consecutive
// channels, so loads and stores are 16 bytes a lane, and the row's mean square and maximum are
// warp reductions over registers.
#include "latent.cuh"

namespace csa {

namespace {

constexpr int kMaxVec = 4; // append: 8-channel vectors per lane, R <= 32 * 8 * 4 = 1024
constexpr double kTwoPi = 6.283185307179586476925287;

__device__ __forceinline__ void ld8(const float *p, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void ld8(const uint16_t *p, float (&v)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The rotation of pair i at position p is by p * base^(-2i/rd).  The angle of a far position needs
// more than 24 bits before its whole turns are taken off, so it is formed and reduced in 64 bits; the
// sine and cosine of what is left are taken in 32.  The frequency of a lane's pair is computed once
// for all rows of the warp.
template <typename Tin> __global__ void __launch_bounds__(256) latent_append_kernel(LatentAppendArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * 8;
    const int rd = a.out.rope_dims, R = a.out.c - rd;
    const double lb = a.base > 0 ? log(a.base) : 0.0;
    double freq = 0.0; // of pair `lane`; further pairs (rd > 64) are formed below
    if (a.base > 0 && 2 * lane < rd) freq = exp(-(2.0 * lane / rd) * lb);
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < a.n; i += warps) {
        const int64_t p = a.pos[i];
        if (p < 0) continue;
        const int64_t b = a.seq ? a.seq[i] : i;
        const int64_t row = b >= 0 && b < a.B ? a.map.row(b, p) : -1;
        if (row < 0) {
            if (lane == 0) flag_error(a.err, CSA_DEVERR_INDEX);
            continue;
        }
        const Tin *x = static_cast<const Tin *>(a.x) + i * a.out.c;
        float v[kMaxVec][8];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxVec; ++k) {
            const int j = 8 * (lane + 32 * k);
            if (j < R) {
                ld8(x + j, v[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[k][e], v[k][e], ss);
            }
        }
        // the rotated part, its loads beside those above
        for (int k = lane; 2 * k < rd; k += 32) {
            float u = ld1<Tin>(x, R + 2 * k), w = ld1<Tin>(x, R + 2 * k + 1);
            if (a.base > 0) {
                const double f = k == lane ? freq : exp(-(2.0 * k / rd) * lb);
                const double ang = (double)p * f;
                float sn, cs;
                sincosf((float)(ang - kTwoPi * rint(ang / kTwoPi)), &sn, &cs);
                const float t = fmaf(u, cs, -w * sn);
                w = fmaf(u, sn, w * cs);
                u = t;
            }
            *reinterpret_cast<uint32_t *>(a.out.rope + row * rd + 2 * k) =
                uint32_t(f32_to_bf16_bits(u)) | (uint32_t(f32_to_bf16_bits(w)) << 16);
        }
        if (a.g) {
            const float f = 1.f / sqrtf(warp_sum(ss) / (float)R + a.eps);
#pragma unroll
            for (int k = 0; k < kMaxVec; ++k) {
                const int j = 8 * (lane + 32 * k);
                if (j < R) {
                    float g[8];
                    ld8(a.g + j, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * f * g[e];
                }
            }
        }
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxVec; ++k)
            if (8 * (lane + 32 * k) < R) {
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[k][e]));
            }
        float sc = __fdiv_rn(warp_max(m), 448.f);
        if (!(sc > 0.f)) sc = 1.f;
#pragma unroll
        for (int k = 0; k < kMaxVec; ++k) {
            const int j = 8 * (lane + 32 * k);
            if (j < R) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e >> 2] |= uint32_t(e4m3_encode(__fdiv_rn(v[k][e], sc))) << (8 * (e & 3));
                *reinterpret_cast<uint2 *>(a.out.fp8 + row * R + j) = make_uint2(w[0], w[1]);
            }
        }
        if (lane == 0) a.out.scale[row] = sc;
    }
}

// 16 FP8 codes times the row scale, stored as bf16 or fp32.
__device__ __forceinline__ void st16(uint16_t *p, const float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = uint32_t(f32_to_bf16_bits(v[8 * h + 2 * e])) | (uint32_t(f32_to_bf16_bits(v[8 * h + 2 * e + 1])) << 16);
        *reinterpret_cast<uint4 *>(p + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void st16(float *p, const float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 4; ++h) *reinterpret_cast<float4 *>(p + 4 * h) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
}

constexpr int kGatherRows = 8; // rows per warp

template <typename Tout> __global__ void __launch_bounds__(256) latent_gather_kernel(LatentGatherArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t n0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kGatherRows;
    const int rd = a.rows.rope_dims, R = a.rows.c - rd;
    // lane l < kGatherRows resolves row n0 + l: -2 outside the runs (left as it is), -1 refused
    int64_t mine = -2;
    if (lane < kGatherRows) {
        const int64_t n = n0 + lane;
        if (n < a.n_out && n >= a.cu[0] && n < a.cu[a.B]) {
            int64_t lo = 0, hi = a.B; // the last b with cu[b] <= n
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (a.cu[mid] <= n) lo = mid;
                else hi = mid;
            }
            const int64_t s = n - a.cu[lo] + (a.start ? a.start[lo] : 0);
            mine = s >= 0 ? a.map.row(lo, s) : -1;
            if (mine < 0) {
                mine = -1;
                flag_error(a.err, CSA_DEVERR_INDEX);
            }
        }
    }
    for (int j0 = 0; a.lat && j0 < R; j0 += 512) { // every lane takes part in the shuffles
        const int j = j0 + 16 * lane;
        uint4 u[kGatherRows];
        float s[kGatherRows];
        int64_t row[kGatherRows];
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            row[r] = __shfl_sync(0xffffffffu, mine, r);
            u[r] = make_uint4(0, 0, 0, 0);
            s[r] = 0.f;
            if (row[r] >= 0 && j < R) {
                u[r] = __ldg(reinterpret_cast<const uint4 *>(a.rows.fp8 + row[r] * R + j));
                s[r] = __ldg(a.rows.scale + row[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
            if (row[r] < -1 || j >= R) continue;
            const uint32_t w[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = e4m3_decode(uint8_t(w[e >> 2] >> (8 * (e & 3)))) * s[r];
            st16(static_cast<Tout *>(a.lat) + (n0 + r) * R + j, v);
        }
    }
    if (a.rope) {
        const int per = rd / 8; // 16-byte vectors a row
        for (int e = lane; e - lane < kGatherRows * per; e += 32) {
            const int r = e / per < kGatherRows ? e / per : kGatherRows - 1;
            const int64_t row = __shfl_sync(0xffffffffu, mine, r);
            if (e >= kGatherRows * per || row < -1) continue;
            const int j = 8 * (e % per);
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row >= 0) ld8(a.rows.rope + row * rd + j, v);
            Tout *dst = static_cast<Tout *>(a.rope) + (n0 + r) * rd + j;
            st4(dst, 0, make_float4(v[0], v[1], v[2], v[3]));
            st4(dst, 4, make_float4(v[4], v[5], v[6], v[7]));
        }
    }
}

} // namespace

cudaError_t launch_latent_append(const LatentAppendArgs &a, int in_dtype, cudaStream_t st)
{
    const int64_t blocks = (a.n + 7) / 8, most = 16 * (int64_t)device_sms();
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    if (in_dtype == CSA_F32) latent_append_kernel<float><<<grid, 256, 0, st>>>(a);
    else latent_append_kernel<uint16_t><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherArgs &a, int out_dtype, cudaStream_t st)
{
    const unsigned grid = (unsigned)((a.n_out + 8 * kGatherRows - 1) / (8 * kGatherRows));
    if (out_dtype == CSA_F32) latent_gather_kernel<float><<<grid, 256, 0, st>>>(a);
    else latent_gather_kernel<uint16_t><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

} // namespace csa
