// latent_generic.cu -- latent attention on the CUDA cores, for the shapes and types that the
// tensor-core kernels do not take, and the merge of a split decode.
//
// Both kernels hold a tile of keys in shared memory as fp32.  Scores: lane = key, the query's
// channels broadcast from shared memory, so a key's dot product needs no reduction over lanes (the
// odd row stride keeps the 32 lanes in 32 banks).  Values: lane = channel (+ 32 i), a key's
// probability by shuffle.  One pass with the running maximum and sum of the softmax (log2 domain,
// fp32).  ALU-bound: (c + R) fused multiply-adds per query row and key.
#include "latent.cuh"

namespace csa {

namespace {

constexpr int kWarps = 8, kRowsPerWarp = 4;
constexpr int kRB = kWarps * kRowsPerWarp; // query rows of a block
constexpr int kKT = 32;                    // keys of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

using Split = LatentSplit<kRB, kKT, 1>;
using TcSplit32 = LatentSplit<32, 128, 4>; // of the tensor-core kernels
using TcSplit64 = LatentSplit<64, 64, 4>;

// One tile of up to 32 keys for one query row: q [dk] and kt [32, ldk] in shared memory, score of
// key `lane` masked by `seen`, values vt[j * ldv + ch], ch < dv.
template <int NV>
__device__ __forceinline__ void tile_step(const float *q, const float *kt, int ldk, int dk, const float *vt, int ldv, int dv,
                                          float scale_log2, bool seen, int lane, float &m, float &l, float (&acc)[NV])
{
    float z = 0.f;
    for (int d = 0; d < dk; ++d) z = fmaf(q[d], kt[lane * ldk + d], z);
    z = seen ? z * scale_log2 : -INFINITY;
    float m_new = fmaxf(m, warp_max(z)); // (of what is a number)
    if (m_new == -INFINITY) {
        if (!__any_sync(0xffffffffu, z != z)) return; // nothing seen so far
        m_new = 0.f; // a score that is none: its p, and with it the row, is NaN
    }
    const float f = exp2f(m - m_new), p = seen ? exp2f(z - m_new) : 0.f;
    m = m_new;
    l = fmaf(l, f, warp_sum(p));
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] *= f;
    for (int j = 0; j < kKT; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p, j);
        if (pj == 0.f) continue; // an unseen key's values are not touched, whatever they are
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < dv) acc[i] = fmaf(pj, vt[j * ldv + lane + 32 * i], acc[i]);
    }
}

// ---- absorbed form -------------------------------------------------------------------------

constexpr int kMaxNV = 16; // R <= 512

__global__ void __launch_bounds__(32 * kWarps) latent_decode_generic_kernel(LatentDecodeArgs a)
{
    extern __shared__ float sm[];
    cudaTriggerProgrammaticLaunchCompletion(); // the merge may come up
    __shared__ int64_t s_at[4];
    __shared__ int ok[kKT];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rd = a.rows.rope_dims, R = a.rows.c - rd, c = a.rows.c, ld = c + 1;
    float *kt = sm, *qs = sm + kKT * ld; // [kKT, ld], [kRB, c]
    if (warp == 0) LatentWalk<Split>::begin(a, lane, s_at);
    __syncthreads();
    LatentWalk<Split> walk(a, s_at);
    LatentRun run;
    while (walk.next(a, run)) {
        const int64_t b = run.b, t0 = run.t0, t1 = run.t1;
        const int rb = run.rb;
        // the block's queries
        const int row0 = rb * kRB, n_rows = min(kRB, a.Lq * a.H - row0);
        __syncthreads();
        for (int e = threadIdx.x; e < n_rows * c; e += 32 * kWarps)
            qs[e] = bf16_to_f32(a.q[((int64_t)b * a.Lq * a.H + row0) * c + e]);
        float m[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][kMaxNV];
#pragma unroll
        for (int u = 0; u < kRowsPerWarp; ++u) {
            m[u] = -INFINITY;
            l[u] = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxNV; ++i) acc[u][i] = 0.f;
        }
        const int64_t seen_all = latent_visible(a, b, a.Lq - 1);
        for (int64_t t = t0; t < t1; ++t) {
            __syncthreads();
            for (int e = threadIdx.x; e < kKT * (c / 4); e += 32 * kWarps) {
                const int j = e / (c / 4), ch = 4 * (e % (c / 4));
                const int64_t s = t * kKT + j;
                const int64_t row = s < seen_all ? a.map.row(b, s) : -1;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0) {
                    if (ch < R) {
                        const uint32_t u = *reinterpret_cast<const uint32_t *>(a.rows.fp8 + row * R + ch);
                        const float sc = a.rows.scale[row];
                        v = make_float4(e4m3_decode(u & 255) * sc, e4m3_decode((u >> 8) & 255) * sc,
                                        e4m3_decode((u >> 16) & 255) * sc, e4m3_decode(u >> 24) * sc);
                    } else {
                        v = Ld4<uint16_t>::at(a.rows.rope, row * rd + (ch - R));
                    }
                }
                float *d = kt + j * ld + ch;
                d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                if (ch == 0) {
                    ok[j] = row >= 0;
                    if (s < seen_all && row < 0) flag_error(a.err, CSA_DEVERR_INDEX);
                }
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kRowsPerWarp; ++u) {
                const int r = warp * kRowsPerWarp + u;
                if (r >= n_rows) continue;
                const bool seen = ok[lane] && t * kKT + lane < latent_visible(a, b, (row0 + r) / a.H);
                tile_step<kMaxNV>(qs + r * c, kt, ld, c, kt, ld, R, a.scale * kLog2e, seen, lane, m[u], l[u], acc[u]);
            }
        }
        const bool first = run.first, whole = run.whole;
#pragma unroll
        for (int u = 0; u < kRowsPerWarp; ++u) {
            const int r = warp * kRowsPerWarp + u;
            if (r >= n_rows) continue;
            if (whole) {
                const int64_t row = (int64_t)b * a.Lq * a.H + row0 + r;
                const float inv = l[u] != 0.f ? 1.f / l[u] : 0.f;
#pragma unroll
                for (int i = 0; i < kMaxNV; ++i)
                    if (lane + 32 * i < R) a.o[row * R + lane + 32 * i] = f32_to_bf16_bits(acc[u][i] * inv);
                if (a.lse && lane == 0) a.lse[row] = l[u] != 0.f ? (m[u] + log2f(l[u])) * kLn2 : -INFINITY;
            } else {
                float *p = latent_part<kRB>(a.part, R, 2 * (int64_t)blockIdx.x + first);
                if (lane == 0) p[2 * r] = m[u], p[2 * r + 1] = l[u];
#pragma unroll
                for (int i = 0; i < kMaxNV; ++i)
                    if (lane + 32 * i < R) p[latent_part_at<kRB>(r, lane + 32 * i)] = acc[u][i];
            }
        }
    }
}

// Merge of the parts of a run that the split cut.  With part i holding the maximum m_i (log2 domain), the sum l_i and the
// unnormalised output O_i, the run's are m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i; the output is
// O / l.  Bound by latency, its own (where the run lies takes some 3 us to find) and that of its loads, of which a thread
// has 8 under way.  Of many parts a CTA takes 4 rows and 128 channels, and up to 4 groups of 128 threads share the
// parts (1 x 64k keys x 16 heads, 148 parts: 12 us behind the parts' kernel; one group 45).  Of few parts of many rows it
// takes 16 rows and all channels, four rows a thread (32 x 256 rows in 2 or 3 parts: 16 us; 4 rows a CTA 33; the
// whole call of 64 x 64 rows after 1k to 4k keys 61 us, 70; but of 64 x 16 rows 45, 43).
constexpr int kMaxParts = 512;

template <class Split, int RB, int ROWS> __global__ void __launch_bounds__(512) latent_merge_kernel(LatentDecodeArgs a)
{
    constexpr int U = ROWS / 4, kLoads = 8 / U, kLanes = ROWS == 4 ? 128 : 512; // rows a thread, parts at a time, threads of a group
    static_assert(RB % ROWS == 0, "a CTA's rows lie in one row block");
    __shared__ int64_t s_at[2];
    __shared__ float red[2][16][ROWS];
    extern __shared__ float4 merge_smem[]; // sums of the groups behind the first, weights and sums of the parts
    const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
    const int rows = a.Lq * a.H, blocks = (rows + ROWS - 1) / ROWS;
    const int64_t b = blockIdx.x / blocks;
    const int r0 = (int)(blockIdx.x % blocks) * ROWS, rb = r0 / RB;
    const int R = a.rows.c - a.rows.rope_dims;
    const int64_t nrb = a.par > 1 ? 1 : Split::row_blocks(a.Lq, a.H), G = a.grid / a.par;
    float4 *sums = merge_smem;
    float *weight = reinterpret_cast<float *>(sums + (blockDim.x - kLanes)), *part_sum = weight + ROWS * G;
    if (tid < 64) { // the length before this sequence (warp 0), from it on (warp 1)
        const int64_t s = tid < 32 ? Split::warp_total(a, 0, b, lane) : Split::warp_total(a, b, a.B, lane);
        if (lane == 0) s_at[tid >> 5] = s * nrb;
    }
    const int64_t length = Split::length(a, b);
    __syncthreads();
    const int64_t T = s_at[0] + s_at[1], begin = s_at[0] + (a.par > 1 ? 0 : rb * length);
    const int64_t s0 = begin + Split::kCost, s1 = begin + length - 1; // the places of its first and last tile
    // the CTAs (or groups) that hold the run's first and last tile: the largest i with floor(i T / G) <= place
    const int64_t i0 = quotient((s0 + 1) * G - 1, T), i1 = quotient((s1 + 1) * G - 1, T);
    // launched beside the kernel that writes the parts: every block waits for it, those with nothing to do too, since
    // what follows in the stream waits for this kernel alone
    cudaGridDependencySynchronize();
    if (i0 == i1) return; // finished by the CTA that holds it
    const int n = (int)(i1 - i0 + 1);
    // part k: slot 2 i + 1 where the run begins, slot 2 i behind; a CTA without tiles has none
    const int64_t cta0 = i0 * a.par + (a.par > 1 ? rb : 0), step = 2 * a.par * latent_part_size<RB>(R);
    const float *first = latent_part<RB>(a.part, R, 2 * cta0 + 1), *rest = latent_part<RB>(a.part, R, 2 * cta0);
    auto part = [&](int k) { return k == 0 ? first : rest + k * step; };
    const int wr = tid % ROWS; // the row that this thread weighs parts of
    auto over_threads = [&](float (&at)[16][ROWS], float v, auto op) { // of those with this row
#pragma unroll
        for (int o = ROWS; o < 32; o <<= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane < ROWS) at[tid >> 5][lane] = v;
        __syncthreads();
        v = at[0][wr];
        for (int w = 1; w < warps; ++w) v = op(v, at[w][wr]);
        return v;
    };
    float m = -INFINITY;
    const int row_at = 2 * ((r0 + wr) % RB), stride = blockDim.x / ROWS;
#pragma unroll 4
    for (int k = tid / ROWS; k < n; k += stride) {
        float2 v = make_float2(-INFINITY, 0.f);
        if (r0 + wr < rows && (T >= G || quotient(T * (i0 + k), G) < quotient(T * (i0 + k + 1), G)))
            v = __ldcg(reinterpret_cast<const float2 *>(part(k) + row_at));
        weight[ROWS * k + wr] = v.x;
        part_sum[ROWS * k + wr] = v.y;
        m = fmaxf(m, v.x);
    }
    m = over_threads(red[0], m, [](float x, float y) { return fmaxf(x, y); });
    float l = 0.f;
    for (int k = tid / ROWS; k < n; k += stride) {
        const float mk = weight[ROWS * k + wr], w = mk == -INFINITY ? 0.f : exp2f(mk - m);
        weight[ROWS * k + wr] = w;
        l = fmaf(w, part_sum[ROWS * k + wr], l);
    }
    l = over_threads(red[1], l, [](float x, float y) { return x + y; }); // (and every weight is there)
    if (tid < ROWS) { // (this thread's row)
        red[0][0][tid] = l != 0.f ? 1.f / l : 0.f;
        if (a.lse && r0 + tid < rows && blockIdx.y == 0) a.lse[b * rows + r0 + tid] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    // every group takes an equal share of the parts
    const int t = tid % kLanes, group = tid / kLanes, groups = blockDim.x / kLanes, k1 = n * (group + 1) / groups;
    const int ch = kLanes * (int)blockIdx.y + 4 * (t >> 2), u0 = t & 3;
    int at[U];
    bool there[U];
    float4 acc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        at[i] = latent_part_at<RB>((r0 + u0 + 4 * i) % RB, ch);
        there[i] = r0 + u0 + 4 * i < rows && ch < R;
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k0 = n * group / groups; k0 < k1; k0 += kLoads) { // 8 loads on their way together
        float4 v[kLoads][U];
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (there[i]) v[e][i] = __ldcg(reinterpret_cast<const float4 *>(part(min(k0 + e, k1 - 1)) + at[i]));
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float w = there[i] && k0 + e < k1 ? weight[ROWS * (k0 + e) + u0 + 4 * i] : 0.f;
                if (w != 0.f) { // else nothing was seen there, or nothing was written
                    acc[i].x = fmaf(w, v[e][i].x, acc[i].x);
                    acc[i].y = fmaf(w, v[e][i].y, acc[i].y);
                    acc[i].z = fmaf(w, v[e][i].z, acc[i].z);
                    acc[i].w = fmaf(w, v[e][i].w, acc[i].w);
                }
            }
    }
    if constexpr (U == 1)
        if (groups > 1) {
            if (group > 0) sums[kLanes * (group - 1) + t] = acc[0];
            __syncthreads();
            if (group > 0) return;
            for (int i = 0; i < groups - 1; ++i) {
                const float4 v = sums[kLanes * i + t];
                acc[0].x += v.x, acc[0].y += v.y, acc[0].z += v.z, acc[0].w += v.w;
            }
        }
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (there[i]) {
            const float inv = red[0][0][u0 + 4 * i];
            st4(a.o, (b * rows + r0 + u0 + 4 * i) * R + ch, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
        }
}

// ---- expanded form -------------------------------------------------------------------------

constexpr int kMaxNVp = 8; // dv <= 256

template <typename T> __global__ void __launch_bounds__(32 * kWarps) latent_prefill_generic_kernel(LatentPrefillArgs a)
{
    extern __shared__ float sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int dk = a.dn + a.dr, ldk = dk + 1, h = blockIdx.y;
    const int64_t per = (a.max_q + kRB - 1) / kRB, b = blockIdx.x / per;
    float *kt = sm, *vt = kt + kKT * ldk, *qs = vt + kKT * a.dv; // [kKT, ldk], [kKT, dv], [kRB, dk]
    int64_t q0, q1, k0, k1;
    packed_range(a.cu_q, b, a.Tq, &q0, &q1);
    packed_range(a.cu_k, b, a.Tk, &k0, &k1);
    const int64_t nq = q1 - q0, nk = k1 - k0, lag = nk - nq;
    const int64_t i0 = (blockIdx.x % per) * kRB;
    if (i0 >= nq || i0 >= a.max_q) return;
    const int n_rows = (int)min((int64_t)kRB, min(nq, a.max_q) - i0);
    const T *q = static_cast<const T *>(a.q), *kv = static_cast<const T *>(a.kv), *kr = static_cast<const T *>(a.k_rope);
    for (int e = threadIdx.x; e < n_rows * dk; e += 32 * kWarps)
        qs[e] = ld1<T>(q, ((q0 + i0 + e / dk) * a.H + h) * dk + e % dk);
    float m[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][kMaxNVp];
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
        m[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxNVp; ++i) acc[u][i] = 0.f;
    }
    const int64_t seen_all = a.causal ? max((int64_t)0, min(nk, i0 + n_rows + lag)) : nk;
    for (int64_t t = 0; t < seen_all; t += kKT) {
        const int n = (int)min((int64_t)kKT, seen_all - t);
        __syncthreads();
        for (int e = threadIdx.x; e < kKT * (dk + a.dv); e += 32 * kWarps) {
            const int j = e / (dk + a.dv), ch = e % (dk + a.dv);
            const int64_t row = k0 + t + j;
            float v = 0.f;
            if (j < n) v = ch >= a.dn && ch < dk ? ld1<T>(kr, row * a.dr + ch - a.dn)
                                                 : ld1<T>(kv, (row * a.H + h) * (a.dn + a.dv) + (ch < a.dn ? ch : ch - a.dr));
            if (ch < dk) kt[j * ldk + ch] = v;
            else vt[j * a.dv + ch - dk] = v;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kRowsPerWarp; ++u) {
            const int r = warp * kRowsPerWarp + u;
            if (r >= n_rows) continue;
            const bool seen = lane < n && (!a.causal || t + lane <= i0 + r + lag);
            tile_step<kMaxNVp>(qs + r * dk, kt, ldk, dk, vt, a.dv, a.dv, a.scale * kLog2e, seen, lane, m[u], l[u], acc[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
        const int r = warp * kRowsPerWarp + u;
        if (r >= n_rows) continue;
        const int64_t row = (q0 + i0 + r) * a.H + h;
        const float inv = l[u] != 0.f ? 1.f / l[u] : 0.f;
#pragma unroll
        for (int i = 0; i < kMaxNVp; ++i) {
            const int ch = lane + 32 * i;
            if (ch >= a.dv) continue;
            if constexpr (sizeof(T) == 4) static_cast<float *>(a.o)[row * a.dv + ch] = acc[u][i] * inv;
            else static_cast<uint16_t *>(a.o)[row * a.dv + ch] = f32_to_bf16_bits(acc[u][i] * inv);
        }
        if (a.lse && lane == 0) a.lse[row] = l[u] != 0.f ? (m[u] + log2f(l[u])) * kLn2 : -INFINITY;
    }
}

} // namespace

size_t latent_decode_generic_workspace(int64_t B, int Lq, int H, int R, int64_t max_len, int *grid, int *par)
{
    Split::plan(B, Lq, H, max_len, device_sms(), grid, par);
    return (size_t)*grid * 2 * latent_part_size<kRB>(R) * sizeof(float);
}

template <class Split, int RB> static cudaError_t launch_merge(const LatentDecodeArgs &a, cudaStream_t st)
{
    if (a.grid == a.par) return cudaSuccess; // one CTA, or one group, cuts no run
    if (a.grid > kMaxParts) return cudaErrorInvalidValue;
    const int64_t parts = (a.grid / a.par + a.B - 1) / a.B; // of a run of the average length
    const bool few = parts <= 8 && a.B * a.Lq * a.H >= 16 * device_sms(); // and rows enough for all SMs
    const int rows = few ? 16 : 4, threads = few || parts > 16 ? 512 : parts > 8 ? 256 : 128, R = a.rows.c - a.rows.rope_dims;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * ((a.Lq * a.H + rows - 1) / rows)), few ? 1u : (unsigned)((R + 127) / 128));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (few ? 0 : (size_t)(threads - 128) * sizeof(float4)) + 2 * (size_t)(a.grid / a.par) * rows * sizeof(float);
    cfg.stream = st;
    // its blocks come up while the parts are written, and wait for them
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, latent_merge_kernel<Split, RB, 16>, a) : cudaLaunchKernelEx(&cfg, latent_merge_kernel<Split, RB, 4>, a);
}

cudaError_t launch_latent_merge_tc(const LatentDecodeArgs &a, int rows, cudaStream_t st)
{
    return rows == 32 ? launch_merge<TcSplit32, 32>(a, st) : launch_merge<TcSplit64, 64>(a, st);
}

// The kernels' limits of shared memory are those of the largest shapes, set once: a limit set for each call would be taken
// from it by a call of another host thread.
constexpr int kMaxC = 640, kMaxDk = 256, kMaxDv = 256;
static constexpr size_t decode_smem(int c) { return (size_t)(kKT * (c + 1) + kRB * c) * sizeof(float); }
static constexpr size_t prefill_smem(int dk, int dv) { return (size_t)(kKT * (dk + 1) + kKT * dv + kRB * dk) * sizeof(float); }

cudaError_t launch_latent_decode_generic(LatentDecodeArgs a, cudaStream_t st)
{
    static std::atomic<bool> done[64];
    const size_t smem = decode_smem(a.rows.c);
    cudaError_t e = prepare_kernel(latent_decode_generic_kernel, decode_smem(kMaxC), 0, done);
    if (e != cudaSuccess) return e;
    latent_decode_generic_kernel<<<(unsigned)a.grid, 32 * kWarps, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_merge<Split, kRB>(a, st);
}

template <typename T> static cudaError_t prefill_generic(const LatentPrefillArgs &a, cudaStream_t st)
{
    static std::atomic<bool> done[64];
    const size_t smem = prefill_smem(a.dn + a.dr, a.dv);
    cudaError_t e = prepare_kernel(latent_prefill_generic_kernel<T>, prefill_smem(kMaxDk, kMaxDv), 0, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.B * ((a.max_q + kRB - 1) / kRB);
    latent_prefill_generic_kernel<T><<<dim3((unsigned)blocks, (unsigned)a.H), 32 * kWarps, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_latent_prefill_generic(const LatentPrefillArgs &a, int dtype, cudaStream_t st)
{
    return dtype == CSA_F32 ? prefill_generic<float>(a, st) : prefill_generic<uint16_t>(a, st);
}

} // namespace csa
