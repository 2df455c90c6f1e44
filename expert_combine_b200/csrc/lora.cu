// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t, :] = base[t, :] + scale_a * (x[t, :] A_a^T) B_a^T,  a = adapter_ids[t]
// with x [T, H], A [L, R, H], B [L, N, R] in BF16 and base/out [T, N] in FP32
// or BF16; a token whose id is outside [0, L) keeps its row of base.
//
// Two products of very different shape: the first ("shrink") reads x and A,
// reduces over H and leaves v [T, R] in FP32; the second ("expand") reads v
// and B, and adds to base over N.  R is small, so both are bound by their
// reads and writes, and by latency when there are few tokens.
//
// Few tokens (decode).  Tokens of one adapter are taken in groups of up to 8
// (the N of an m16n8k16 MMA, the adapter's 16 ranks its M): the CTAs of token t
// work on the group that t leads, i.e. whose earlier tokens of the same adapter
// number a multiple of 8, and the CTAs of the other tokens leave at once.  Every
// CTA finds that out for itself from the ids (one ballot per warp), so nothing
// is sorted beforehand.  Operands come straight from memory into the MMA's
// registers: which k a lane's registers stand for is free as long as A and x
// agree, so a lane takes 8 consecutive k of its row as one 16-byte load, and
// two MMAs use up the four words of each.  The warps of a CTA and the CTAs of a
// group split H; each CTA writes its partial v, and the expand kernel adds the
// partials in order (no atomics), scales them once, and holds one group's v in
// shared memory while each thread forms two columns with FP32 multiply-adds.
#include "internal.h"
#include "common.cuh"

namespace mb {

namespace {

constexpr int kLoraThreads = 256;          // shrink CTA; also the tokens one launch looks at
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraGroup = 8;              // tokens per group
constexpr int kLoraExpThreads = 128;
constexpr int kLoraExpCols = 2 * kLoraExpThreads;

struct LoraArgs {
    const uint16_t* x;        // [T, H]
    const uint16_t* a;        // [L, R, H]
    const uint16_t* b;        // [L, N, R]
    const int32_t* ids;       // [T]
    const float* scales;      // [L] or NULL
    const void* base;         // [T, N]
    void* out;                // [T, N]
    float* part;              // [splits][T][R]
    int T, H, N, R, L;
    int splits, kc;           // H is cut into `splits` runs of kc
};

// The group that token t leads: its members in order (s_member) and their
// number, or 0 when t leads none.  Every thread of the CTA calls it (at least T
// threads' worth of warps in steps); *id is t's adapter, -1 for none.
template <int THREADS>
__device__ __forceinline__ int lora_group(const LoraArgs& a, int t, int* id, uint32_t* s_mask, int* s_member) {
    const int my = a.ids[t];
    *id = my >= 0 && my < a.L ? my : -1;
    if (*id < 0) return 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = warp; w < kLoraThreads / 32; w += THREADS / 32) {
        const int i = w * 32 + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, i < a.T && a.ids[i] == my);
        if (lane == 0) s_mask[w] = m;
    }
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (t >> 5); ++w) before += __popc(s_mask[w]);
    before += __popc(s_mask[t >> 5] & ((1u << (t & 31)) - 1u));
    if (before % kLoraGroup != 0) return 0;
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = t >> 5; w < kLoraThreads / 32 && n < kLoraGroup; ++w) {
            uint32_t m = s_mask[w];
            if (w == (t >> 5)) m &= ~((1u << (t & 31)) - 1u);
            for (; m != 0 && n < kLoraGroup; m &= m - 1) s_member[n++] = w * 32 + __ffs(m) - 1;
        }
        for (int j = n; j < kLoraGroup; ++j) s_member[j] = -1;
        s_member[kLoraGroup] = n;
    }
    __syncthreads();
    return s_member[kLoraGroup];
}

__device__ __forceinline__ void mma_16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shrink of one group and one run of H; MT tiles of 16 ranks.
template <int MT>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_few_kernel(const LoraArgs a) {
    __shared__ uint32_t s_mask[kLoraThreads / 32];
    __shared__ int s_member[kLoraGroup + 1];
    __shared__ float s_v[kLoraWarps][MT * 16][kLoraGroup];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    griddep_wait();
    griddep_launch();
    int id;
    const int n = lora_group<kLoraThreads>(a, t, &id, s_mask, s_member);
    if (n == 0) return;

    const int g = lane >> 2, c = lane & 3;
    const int k_end = min((static_cast<int>(blockIdx.y) + 1) * a.kc, a.H);
    const int tok = s_member[g];
    const uint16_t* xr = a.x + static_cast<size_t>(tok < 0 ? 0 : tok) * a.H;
    const uint16_t* ar = a.a + (static_cast<size_t>(id) * a.R + g) * a.H;
    float acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int k = blockIdx.y * a.kc + warp * 32 + c * 8; k - c * 8 < k_end; k += kLoraWarps * 32) {
        const bool in = k < k_end;
        const uint4 xv = in && tok >= 0 ? ld_nc_v4(xr + k) : zero;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint4 lo = in && 16 * m + g < a.R ? ld_nc_v4(ar + static_cast<size_t>(16 * m) * a.H + k) : zero;
            const uint4 hi =
                in && 16 * m + g + 8 < a.R ? ld_nc_v4(ar + static_cast<size_t>(16 * m + 8) * a.H + k) : zero;
            mma_16n8k16(acc[m], lo.x, hi.x, lo.y, hi.y, xv.x, xv.y);
            mma_16n8k16(acc[m], lo.z, hi.z, lo.w, hi.w, xv.z, xv.w);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        s_v[warp][16 * m + g][2 * c] = acc[m][0];
        s_v[warp][16 * m + g][2 * c + 1] = acc[m][1];
        s_v[warp][16 * m + g + 8][2 * c] = acc[m][2];
        s_v[warp][16 * m + g + 8][2 * c + 1] = acc[m][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * a.R; i += kLoraThreads) {
        const int j = i / a.R, r = i % a.R;
        float v = s_v[0][r][j];
#pragma unroll
        for (int w = 1; w < kLoraWarps; ++w) v += s_v[w][r][j];
        a.part[(static_cast<size_t>(blockIdx.y) * a.T + s_member[j]) * a.R + r] = v;
    }
}

template <typename O>
__device__ __forceinline__ float2 load2(const void* p, size_t i);
template <>
__device__ __forceinline__ float2 load2<float>(const void* p, size_t i) {
    return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
}
template <>
__device__ __forceinline__ float2 load2<uint16_t>(const void* p, size_t i) {
    return unpack_bf16x2(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i));
}
template <typename O>
__device__ __forceinline__ void store2(void* p, size_t i, float2 v);
template <>
__device__ __forceinline__ void store2<float>(void* p, size_t i, float2 v) {
    *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = v;
}
template <>
__device__ __forceinline__ void store2<uint16_t>(void* p, size_t i, float2 v) {
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + i) = pack_bf16x2_rn(v);
}

// Two columns of G tokens: base + v B^T, v [G][R] in shared memory.
template <int G, typename O>
__device__ __forceinline__ void lora_columns(const LoraArgs& a, const float* v, const int* member, int n,
                                             const uint16_t* b, int col) {
    float2 base[G], acc[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        base[j] = j < n ? load2<O>(a.base, static_cast<size_t>(member[j]) * a.N + col) : make_float2(0.0f, 0.0f);
        acc[j] = make_float2(0.0f, 0.0f);
    }
    for (int r = 0; r < a.R; r += 8) {
        const uint4 b0 = ld_nc_v4(b + r), b1 = ld_nc_v4(b + a.R + r);
        const uint32_t w0[4] = {b0.x, b0.y, b0.z, b0.w}, w1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 p0 = unpack_bf16x2(w0[2 * h]), q0 = unpack_bf16x2(w0[2 * h + 1]);
            const float2 p1 = unpack_bf16x2(w1[2 * h]), q1 = unpack_bf16x2(w1[2 * h + 1]);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(v + j * a.R + r + 4 * h);
                acc[j] = fma2(make_float2(f.x, f.x), make_float2(p0.x, p1.x), acc[j]);
                acc[j] = fma2(make_float2(f.y, f.y), make_float2(p0.y, p1.y), acc[j]);
                acc[j] = fma2(make_float2(f.z, f.z), make_float2(q0.x, q1.x), acc[j]);
                acc[j] = fma2(make_float2(f.w, f.w), make_float2(q0.y, q1.y), acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < G; ++j)
        if (j < n) store2<O>(a.out, static_cast<size_t>(member[j]) * a.N + col, add2(base[j], acc[j]));
}

template <typename O>
__global__ void __launch_bounds__(kLoraExpThreads) lora_expand_few_kernel(const LoraArgs a) {
    __shared__ uint32_t s_mask[kLoraThreads / 32];
    __shared__ int s_member[kLoraGroup + 1];
    __shared__ __align__(16) float s_v[kLoraGroup * kMaxLoraRank];
    const int t = blockIdx.x;
    const int col = blockIdx.y * kLoraExpCols + 2 * threadIdx.x;
    griddep_launch();
    // the ids and base were complete before the shrink kernel started; only its partial v is waited for
    int id;
    const int n = lora_group<kLoraExpThreads>(a, t, &id, s_mask, s_member);
    griddep_wait();
    if (n == 0) {
        if (id < 0 && a.out != a.base && col < a.N) {
            const size_t i = static_cast<size_t>(t) * a.N + col;
            store2<O>(a.out, i, load2<O>(a.base, i));
        }
        return;
    }
    const float scale = a.scales != nullptr ? a.scales[id] : 1.0f;
    for (int i = threadIdx.x; i < kLoraGroup * a.R; i += kLoraExpThreads) {
        const int j = i / a.R, r = i % a.R;
        float v = 0.0f;
        if (j < n) {
            const float* p = a.part + static_cast<size_t>(s_member[j]) * a.R + r;
            const size_t pitch = static_cast<size_t>(a.T) * a.R;
            for (int s = 0; s < a.splits; ++s) v += __ldcg(p + s * pitch);
        }
        s_v[i] = v * scale;
    }
    __syncthreads();
    if (col >= a.N) return;
    const uint16_t* b = a.b + (static_cast<size_t>(id) * a.N + col) * a.R;
    if (n <= 2)
        lora_columns<2, O>(a, s_v, s_member, n, b, col);
    else
        lora_columns<kLoraGroup, O>(a, s_v, s_member, n, b, col);
}

// Runs of H per group: enough CTAs for the card when every token leads a
// group, at least 256 (one 32-wide step per warp) of H each.
int lora_splits(int T, int H) {
    int s = 2048 / (T < 1 ? 1 : T);
    if (s > 32) s = 32;
    if (s < 8) s = 8;
    const int most = (H + 255) / 256;
    return s > most ? most : s;
}

template <typename F>
cudaError_t lora_launch(F* kernel, dim3 grid, int threads, const LoraArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t lora_workspace_bytes(int T, int H, int N, int R, int L) {
    const int n = T < kLoraThreads ? T : kLoraThreads;
    return static_cast<size_t>(lora_splits(n, H)) * n * R * sizeof(float);
}

cudaError_t launch_lora_add(const LoraLaunch& l, cudaStream_t s) {
    const size_t size = l.bf16 ? 2 : 4;
    for (int t0 = 0; t0 < l.T; t0 += kLoraThreads) {
        LoraArgs a{};
        a.T = l.T - t0 < kLoraThreads ? l.T - t0 : kLoraThreads;
        a.H = l.H, a.N = l.N, a.R = l.R, a.L = l.L;
        a.x = l.x + static_cast<size_t>(t0) * l.H;
        a.a = l.a, a.b = l.b, a.scales = l.scales;
        a.ids = l.ids + t0;
        a.base = static_cast<const uint8_t*>(l.base) + static_cast<size_t>(t0) * l.N * size;
        a.out = static_cast<uint8_t*>(l.out) + static_cast<size_t>(t0) * l.N * size;
        a.part = static_cast<float*>(l.workspace);
        a.splits = lora_splits(l.T < kLoraThreads ? l.T : kLoraThreads, l.H);
        a.kc = ((l.H + a.splits - 1) / a.splits + 31) / 32 * 32;
        a.splits = (l.H + a.kc - 1) / a.kc;
        const dim3 grid(a.T, a.splits);
        cudaError_t e;
        if (l.R <= 16)
            e = lora_launch(lora_shrink_few_kernel<1>, grid, kLoraThreads, a, s);
        else if (l.R <= 32)
            e = lora_launch(lora_shrink_few_kernel<2>, grid, kLoraThreads, a, s);
        else if (l.R <= 64)
            e = lora_launch(lora_shrink_few_kernel<4>, grid, kLoraThreads, a, s);
        else
            e = lora_launch(lora_shrink_few_kernel<8>, grid, kLoraThreads, a, s);
        if (e != cudaSuccess) return e;
        const dim3 egrid(a.T, (l.N + kLoraExpCols - 1) / kLoraExpCols);
        e = l.bf16 ? lora_launch(lora_expand_few_kernel<uint16_t>, egrid, kLoraExpThreads, a, s)
                   : lora_launch(lora_expand_few_kernel<float>, egrid, kLoraExpThreads, a, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mb
