// C ABI of the masked attention (sigattn_fwd_span, sigattn_bwd_span,
// sigattn_mask_spans in include/sigattn.h).
#include <algorithm>
#include <cmath>

#include "span_fp32.cuh"
#include "span_launch.cuh"

namespace {

using namespace sigattn;

struct SpanArgs {
    const int32_t *seqlens, *spans;
    int Z, L, H, Hk, D;
    float alpha, bias;
    const float *bias_z;
    float cap;
    const float *slopes;
    sigattn_dtype dtype;
};

int64_t tiles_of(int L) { return (static_cast<int64_t>(L) + 127) / 128; }

sigattn_status check_span(const SpanArgs &a, bool *empty) {
    if (a.Z < 0 || a.L < 0 || a.H < 0 || a.Hk < 0) return SIGATTN_ERR_INVALID_ARG;
    if (a.D != 64 && a.D != 128) return SIGATTN_ERR_UNSUPPORTED_HEADDIM;
    if (a.dtype != SIGATTN_BF16 && a.dtype != SIGATTN_FP32) return SIGATTN_ERR_UNSUPPORTED_DTYPE;
    if (a.H > 65535 || a.Z > 65535 || a.L > INT_MAX - 256) return SIGATTN_ERR_INVALID_ARG;
    if (!(a.cap >= 0.0f) || !std::isfinite(a.cap) ||
        (a.cap > 0.0f && !std::isfinite(a.alpha / a.cap)))
        return SIGATTN_ERR_INVALID_ARG;
    if (a.H == 0 && a.Hk != 0) return SIGATTN_ERR_INVALID_ARG;    // dK, dV would have no query
    *empty = a.Z == 0 || a.L == 0 || a.H == 0;
    if (*empty) return SIGATTN_OK;
    if (a.Hk == 0 || a.H % a.Hk != 0) return SIGATTN_ERR_INVALID_ARG;
    if (a.seqlens == nullptr) return SIGATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a.spans) & 7u) != 0) return SIGATTN_ERR_MISALIGNED;
    // the grid of the fp32 path
    if (a.dtype == SIGATTN_FP32 &&
        (static_cast<int64_t>(a.L) + kF32Rows - 1) / kF32Rows * a.Z > int64_t(INT_MAX) / (a.H + a.Hk))
        return SIGATTN_ERR_TOO_LARGE;
    return SIGATTN_OK;
}

SpanKind kind_of(const SpanArgs &a) {
    return SpanKind{a.D, g_sigmoid_mode.load(), score_terms(a.cap, a.slopes)};
}

SpanSource source_of(const SpanArgs &a, int *status) {
    return SpanSource{reinterpret_cast<const int2 *>(a.spans), a.seqlens, a.L, status};
}

SpanF32Params f32_params(const SpanArgs &a, int *status) {
    SpanF32Params p = {};
    p.src = source_of(a, status);
    p.Z = a.Z;
    p.H = a.H;
    p.Hk = a.Hk;
    p.group = a.H / a.Hk;
    p.alpha = a.alpha;
    p.bias = a.bias;
    p.cap = a.cap;
    p.bias_z = a.bias_z;
    p.slopes = a.slopes;
    return p;
}

// Whether a kernel's blocks start tile by tile over all heads of a sample (the
// tiles with the most work first) instead of head by head: when what they stream
// (`tensors` of them, per key head) fits L2 with room to spare, so that nothing
// is read twice from memory.
constexpr int64_t kStreamMost = int64_t(64) << 20;
bool heads_first(const SpanArgs &a, int tensors, int64_t tiles) {
    return tiles <= 65535 && static_cast<int64_t>(tensors) * a.Z * a.L * a.Hk * a.D * 2 <= kStreamMost;
}

// Blocks that share a tile (span_split.cuh): doubled while the grid stays within
// `most` blocks and each block keeps four of the `steps` that a tile can have.  In us,
// unsplit against split, causal:
//   forward, most = what fits the device at once: 1 x 8192 tokens, 2 heads, D = 128
//     126 -> 73, D = 64 81 -> 52; 1 x 4096 67 -> 29, 44 -> 21.  Beyond that it loses: 96 tiles
//     of at most 16 steps in twos 39.7 -> 35.6, but packed documents 23.9 -> 34.5;
//   dK/dV, the same where heads are shared (a tile then has at least a step per head),
//     twice that from eight to a key head: 1 x 2048, 12 over 2 heads 156 -> 57 (D = 128),
//     197 -> 60 (D = 64); 1 x 8192, 16 over 2 842 -> 745, 1018 -> 567.  Alone in its heads
//     a block leaves SMs to dQ, and more than a block an SM loses (64 tiles at D = 64 in
//     fours 71 -> 81, in twos 70);
//   dQ, a block an SM: 1 x 4096, 2 heads 54 -> 46 (D = 128), 69 -> 46 (D = 64).
unsigned split_of(int64_t blocks, int64_t most, int64_t steps) {
    unsigned c = 1;
    while (c < kMostSplit && blocks * c * 2 <= most && steps >= int64_t(8) * c) c *= 2;
    return c;
}

// blocks of kF32Rows rows of one head
unsigned f32_blocks(const SpanArgs &a, int heads) {
    return static_cast<unsigned>((static_cast<int64_t>(a.L) + kF32Rows - 1) / kF32Rows * heads * a.Z);
}

// Calls f.template operator()<D, G>(): the fp32 kernels with G groups of warps to a
// block.  Few blocks, or the backward of shared heads, whose blocks of keys run
// through all of a key head's queries, are bound by a block's length: backward, D = 64,
// 2 x 128 tokens, 2 heads, slopes, 14.4 -> 12.3 us with four groups, 4 x 200 causal, 16
// over 4 heads 229 -> 201.  Many blocks fill the device without (4 x 200 causal, 12 heads,
// 130 -> 151 us with them).
template <typename F>
sigattn_status with_groups(const SpanArgs &a, int64_t blocks, int sms, bool backward, F &&f) {
    const bool many = a.L <= kF32Chunk || (blocks > int64_t(4) * sms && !(backward && a.H > a.Hk));
    if (a.D == 64) return many ? f.template operator()<64, 1>() : f.template operator()<64, 4>();
    return many ? f.template operator()<128, 1>() : f.template operator()<128, 2>();
}

// The device's state, for a dtype the device can run.
sigattn_status span_device(const SpanArgs &a, int *dev, int **status) {
    int cc = 0;
    sigattn_status s = device_state(dev, &cc, status);
    if (s != SIGATTN_OK) return s;
    if (a.dtype == SIGATTN_BF16) {
        if (cc != 100) return SIGATTN_ERR_UNSUPPORTED_DEVICE;
        return get_encoder();
    }
    return SIGATTN_OK;
}

// Token i of sample z -> the interval of keys it sees.  One block per sample:
// a forward scan of each token's run start (docs), then a backward scan of its
// run end and the rest of the mask.
constexpr int kSpanThreads = 1024;

// Inclusive scan over the block (max, or min when MIN), thread order ascending.
template <bool MIN>
__device__ int block_scan(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = MIN ? min(v, u) : max(v, u);
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = MIN ? min(v, warp_sums[w]) : max(v, warp_sums[w]);
    return v;
}

__global__ void __launch_bounds__(kSpanThreads)
    mask_spans_kernel(SpanSource src, const int *prefix, const int *docs, int causal, int window, int2 *out) {
    __shared__ int part[kSpanThreads / 32];
    __shared__ int carry;
    const int z = blockIdx.x, L = src.L;
    const int n = span_tokens(src, z);
    int2 *row = out + static_cast<size_t>(z) * L;
    const int *doc = docs != nullptr ? docs + static_cast<size_t>(z) * L : nullptr;
    if (threadIdx.x == 0) carry = 0;
    for (int i0 = 0; i0 < L; i0 += kSpanThreads) {
        const int i = i0 + threadIdx.x;
        int start = 0;
        if (doc != nullptr) {
            const bool edge = i < n && i > 0 && doc[i] != doc[i - 1];
            __syncthreads();   // carry of the chunk before
            start = max(block_scan<false>(edge ? i : 0, part), carry);
            __syncthreads();
            if (threadIdx.x == kSpanThreads - 1) carry = start;
        }
        if (i < L) row[i].x = start;
    }
    const int pre = prefix != nullptr ? min(max(prefix[z], 0), L) : 0;
    __syncthreads();
    if (threadIdx.x == 0) carry = n;
    const int chunks = (L + kSpanThreads - 1) / kSpanThreads;
    for (int c = chunks - 1; c >= 0; --c) {
        const int i = c * kSpanThreads + (kSpanThreads - 1 - static_cast<int>(threadIdx.x));
        int end = n;
        if (doc != nullptr) {
            const bool edge = i + 1 < n && doc[i] != doc[i + 1];
            __syncthreads();
            end = min(block_scan<true>(edge ? i + 1 : INT_MAX, part), carry);
            __syncthreads();
            if (threadIdx.x == kSpanThreads - 1) carry = end;
        }
        if (i >= L) continue;
        int lo = row[i].x, hi = end;
        if (causal) hi = min(hi, max(i + 1, prefix != nullptr ? lo + min(pre, L - lo) : 0));
        if (window > 0) {
            lo = max(lo, i - window + 1);
            if (!causal) hi = min(hi, i + min(window, L - i));
        }
        row[i] = i < n && lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
    }
}

}  // namespace

extern "C" {

sigattn_status sigattn_fwd_span(const void *q, const void *k, const void *v, void *o, const int32_t *seqlens,
                                const int32_t *spans, int Z, int L, int H, int Hk, int D, float alpha, float bias,
                                const float *bias_z, float cap, const float *slopes, sigattn_dtype dtype,
                                void *stream) {
    const SpanArgs a{seqlens, spans, Z, L, H, Hk, D, alpha, bias, bias_z, cap, slopes, dtype};
    bool empty = false;
    sigattn_status s = check_span(a, &empty);
    if (s != SIGATTN_OK || empty) return s;
    if (q == nullptr || k == nullptr || v == nullptr || o == nullptr) return SIGATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return SIGATTN_ERR_MISALIGNED;
    int dev = 0, *status = nullptr;
    if ((s = span_device(a, &dev, &status)) != SIGATTN_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SIGATTN_FP32) {
        SpanF32Params p = f32_params(a, status);
        p.q = static_cast<const float *>(q);
        p.k = static_cast<const float *>(k);
        p.v = static_cast<const float *>(v);
        p.o = static_cast<float *>(o);
        const unsigned blocks = f32_blocks(a, H);
        return with_groups(a, blocks, g_sm_count[dev], false, [&]<int D_, int G>() {
            return launch(span_f32_fwd_kernel<D_, G>, dim3(blocks), dim3(SpanF32Smem<D_, G>::kThreads),
                          sizeof(SpanF32Smem<D_, G>), st, p);
        });
    }
    CUtensorMap mq, mk, mv;
    if ((s = encode_bf16_map_uncached(&mq, q, Z, L, H, D)) != SIGATTN_OK) return s;
    if ((s = encode_bf16_map_uncached(&mk, k, Z, L, Hk, D)) != SIGATTN_OK) return s;
    if ((s = encode_bf16_map_uncached(&mv, v, Z, L, Hk, D)) != SIGATTN_OK) return s;
    SpanFwdParams p = {};
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.src = source_of(a, status);
    p.H = H;
    p.group = H / Hk;
    p.alpha = alpha;
    p.bias = bias;
    p.cap = cap;
    p.bias_z = bias_z;
    p.slopes = slopes;
    p.timeout_ns = g_timeout_ns.load();
    const int per = D == 64 ? SpanTiles<64>::N : SpanTiles<128>::N;
    const unsigned pairs = static_cast<unsigned>((tiles_of(L) + per - 1) / per);
    p.heads_first = heads_first(a, 2, pairs);
    p.split = split_of(static_cast<int64_t>(pairs) * H * Z, int64_t(g_sm_count[dev]) * (2 / per), tiles_of(L));
    return launch_span_fwd(kind_of(a), p.heads_first ? dim3(H * p.split, pairs, Z) : dim3(pairs * p.split, H, Z), mq, mk, mv,
                           p, st);
}

size_t sigattn_bwd_span_workspace_bytes(int Z, int L, sigattn_dtype dtype) {
    if (Z <= 0 || L <= 0 || dtype != SIGATTN_BF16) return 0;
    return static_cast<size_t>(Z) * tiles_of(L) * (128 * sizeof(int2) + sizeof(int4));
}

sigattn_status sigattn_bwd_span(const void *q, const void *k, const void *v, const void *dout, void *dq, void *dk,
                                void *dv, const int32_t *seqlens, const int32_t *spans, int Z, int L, int H, int Hk,
                                int D, float alpha, float bias, const float *bias_z, float cap, const float *slopes,
                                void *workspace, size_t workspace_bytes, sigattn_dtype dtype, void *stream) {
    const SpanArgs a{seqlens, spans, Z, L, H, Hk, D, alpha, bias, bias_z, cap, slopes, dtype};
    bool empty = false;
    sigattn_status s = check_span(a, &empty);
    if (s != SIGATTN_OK || empty) return s;
    for (const void *t : {q, k, v, dout, static_cast<const void *>(dq), static_cast<const void *>(dk),
                          static_cast<const void *>(dv)}) {
        if (t == nullptr) return SIGATTN_ERR_INVALID_ARG;
        if (!aligned16(t)) return SIGATTN_ERR_MISALIGNED;
    }
    const size_t need = sigattn_bwd_span_workspace_bytes(Z, L, dtype);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SIGATTN_ERR_INVALID_ARG;
    if (need > 0 && !aligned16(workspace)) return SIGATTN_ERR_MISALIGNED;
    int dev = 0, *status = nullptr;
    if ((s = span_device(a, &dev, &status)) != SIGATTN_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == SIGATTN_FP32) {
        SpanF32Params p = f32_params(a, status);
        p.q = static_cast<const float *>(q);
        p.k = static_cast<const float *>(k);
        p.v = static_cast<const float *>(v);
        p.dout = static_cast<const float *>(dout);
        p.dq = static_cast<float *>(dq);
        p.dk = static_cast<float *>(dk);
        p.dv = static_cast<float *>(dv);
        const unsigned rows = f32_blocks(a, H);
        const unsigned blocks = rows + f32_blocks(a, Hk);
        return with_groups(a, blocks, g_sm_count[dev], true, [&]<int D_, int G>() {
            return launch(span_f32_bwd_kernel<D_, G>, dim3(blocks), dim3(SpanF32Smem<D_, G>::kThreads),
                          sizeof(SpanF32Smem<D_, G>), st, p, rows);
        });
    }
    CUtensorMap mq, mk, mv, mdo;
    if ((s = encode_bf16_map_uncached(&mq, q, Z, L, H, D)) != SIGATTN_OK) return s;
    if ((s = encode_bf16_map_uncached(&mk, k, Z, L, Hk, D)) != SIGATTN_OK) return s;
    if ((s = encode_bf16_map_uncached(&mv, v, Z, L, Hk, D)) != SIGATTN_OK) return s;
    if ((s = encode_bf16_map_uncached(&mdo, dout, Z, L, H, D)) != SIGATTN_OK) return s;
    const unsigned tiles = static_cast<unsigned>(tiles_of(L));
    int4 *hull = static_cast<int4 *>(workspace);
    int2 *clean = reinterpret_cast<int2 *>(hull + static_cast<size_t>(Z) * tiles);
    SpanBwdParams p = {};
    p.dq = static_cast<__nv_bfloat16 *>(dq);
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.src = source_of(a, status);
    p.H = H;
    p.Hk = Hk;
    p.group = H / Hk;
    p.alpha = alpha;
    p.bias = bias;
    p.cap = cap;
    p.bias_z = bias_z;
    p.slopes = slopes;
    p.clean = clean;
    p.hull = hull;
    p.timeout_ns = g_timeout_ns.load();
    if ((s = launch(span_prep_kernel, dim3(tiles, Z), dim3(128), 0, st, p.src, clean, hull)) != SIGATTN_OK) return s;
    // dK/dV first: its blocks are the longer ones (a key head's queries of all its
    // heads), and dQ's fill in behind them
    p.heads_first = heads_first(a, 2 * p.group, tiles);
    const int64_t sms = g_sm_count[dev], slots = sms * (D == 64 ? 2 : 1), key_tiles = static_cast<int64_t>(tiles) * Hk * Z;
    p.split = split_of(key_tiles, p.group == 1 ? sms : p.group < 8 ? slots : 2 * slots, static_cast<int64_t>(tiles) * p.group);
    s = launch_span_dkdv(kind_of(a), p.heads_first ? dim3(Hk * p.split, tiles, Z) : dim3(tiles * p.split, Hk, Z), mq, mk, mv,
                         mdo, p, st);
    if (s != SIGATTN_OK) return s;
    p.heads_first = heads_first(a, 2, tiles);
    p.split = split_of(static_cast<int64_t>(tiles) * H * Z, sms, tiles);
    return launch_span_dq(kind_of(a), p.heads_first ? dim3(H * p.split, tiles, Z) : dim3(tiles * p.split, H, Z), mq, mk, mv,
                          mdo, p, st);
}

sigattn_status sigattn_mask_spans(const int32_t *seqlens, const int32_t *prefix, const int32_t *docs, int causal,
                                  int window, int Z, int L, int32_t *spans, void *stream) {
    if (Z < 0 || L < 0 || Z > 65535 || L > INT_MAX - 2 * kSpanThreads || window < 0) return SIGATTN_ERR_INVALID_ARG;
    if (prefix != nullptr && (!causal || window > 0)) return SIGATTN_ERR_INVALID_ARG;
    if (Z == 0 || L == 0) return SIGATTN_OK;
    if (seqlens == nullptr || spans == nullptr) return SIGATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(spans) & 7u) != 0) return SIGATTN_ERR_MISALIGNED;
    int dev = 0, cc = 0, *status = nullptr;
    sigattn_status s = device_state(&dev, &cc, &status);
    if (s != SIGATTN_OK) return s;
    return launch(mask_spans_kernel, dim3(Z), dim3(kSpanThreads), 0, static_cast<cudaStream_t>(stream),
                  SpanSource{nullptr, seqlens, L, status}, prefix, docs, causal, std::min(window, L),
                  reinterpret_cast<int2 *>(spans));
}

}  // extern "C"
