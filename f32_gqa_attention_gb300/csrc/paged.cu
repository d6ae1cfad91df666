// paged.cu -- the small operators of the paged cache: page maps, plans of
// drafted trees, op "rope" at given positions and op "cache_write" through a
// slot map (op catalog, vtmu.mpakt.dev/api/ops, for the two ops' arithmetic).
#include "paged.cuh"
#include "paged_kernels.h"
#include "rope.cuh"

namespace vtmu {
namespace {

constexpr int64_t kWave = 152 * 8;  // CTAs of 256 threads that are resident at once

// ---- page_map -------------------------------------------------------------------
// Request b needs want_b - held_b new pages, want = ceil((len + added) / P) and
// held = ceil(len / P), both at most max_pages; page k of the call (k counted
// over the requests in order) is free[n_free - 1 - k].  Every CTA adds up the
// needs of the requests before its own by itself (a few loads per thread), so
// that one launch with no ordering between CTAs does: a CTA never reads a table
// entry that another one writes, new pages being read off the stack.  CTA
// (b, y) serves every gridDim.y-th chunk of request b's rows; the CTAs of b ==
// requests clear the rows before the first request and behind the last one.  Bound
// by the launch: the accepted rows of 7 trees and 256 prompts of 1 to 1021 rows take
// the same 25 us from the host; 3.1-3.9 and 6.6-7.3 us a call in a replayed graph.
constexpr int kMapThreads = 256;

struct Need {
    int64_t len, added, held, want;
};
__device__ __forceinline__ Need page_need(const PageMapArgs& a, const RowRange& all, int b) {
    Need n;
    const PackedRows r = packed_rows(a.cu_rows, b, all, a.rows);
    n.len = max(__ldg(a.lens + b), 0);
    n.added = r.n;
    if (a.accept) {
        const uint64_t inside = r.n >= 64 ? ~0ull : (1ull << r.n) - 1;
        n.added = __popcll(__ldg(reinterpret_cast<const unsigned long long*>(a.accept) + b) & inside);
    }
    n.held = min((n.len + a.page_size - 1) / a.page_size, (int64_t)a.max_pages);
    n.want = min((n.len + n.added + a.page_size - 1) / a.page_size, (int64_t)a.max_pages);
    return n;
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const PageMapArgs a) {
    __shared__ long long s_sum[kMapThreads / 32];
    const int b = blockIdx.x;
    const int64_t step = (int64_t)gridDim.y * kMapThreads, at = (int64_t)blockIdx.y * kMapThreads + threadIdx.x;
    const RowRange all = rows_of_all(a.cu_rows, a.requests, a.rows);
    // Pages taken by the requests before b (by all of them for b == requests).
    long long before = 0;
    for (int i = threadIdx.x; i < b; i += kMapThreads) {
        const Need n = page_need(a, all, i);
        before += n.want - n.held;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < kMapThreads / 32; ++w) before += s_sum[w];
    const int64_t n_free = clamp64(__ldg(a.n_free), 0, a.free_capacity);

    if (b == a.requests) {
        if (at == 0) *a.n_free_out = (int32_t)clamp64(n_free - before, INT32_MIN, INT32_MAX);
        auto clear = [&](int64_t from, int64_t to) {
            for (int64_t r = from + at; r < to; r += step) {
                a.slots[r] = -1;
                if (a.positions) a.positions[r] = -1;
            }
        };
        clear(0, all.first);
        clear(all.last, a.rows);
        return;
    }
    const Need n = page_need(a, all, b);
    const PackedRows r = packed_rows(a.cu_rows, b, all, a.rows);
    int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    auto new_page = [&](int64_t col) -> int32_t {  // col in [held, want)
        const int64_t k = before + col - n.held;
        return k < n_free ? __ldg(a.free_pages + (n_free - 1 - k)) : -1;
    };
    for (int64_t col = n.held + at; col < n.want; col += step) table[col] = new_page(col);
    if (at == 0) a.new_lens[b] = (int32_t)min(n.len + n.added, (int64_t)INT32_MAX);
    const uint64_t keep = a.accept ? __ldg(reinterpret_cast<const unsigned long long*>(a.accept) + b) : 0;
    for (int64_t j = at; j < r.n; j += step) {
        int64_t rank = j;
        bool live = true;
        if (a.accept) {
            live = j < 64 && ((keep >> (j & 63)) & 1);
            rank = __popcll(keep & ((1ull << (j & 63)) - 1));
        }
        const int64_t pos = n.len + rank, col = pos / a.page_size;
        int64_t slot = -1;
        if (live && col < n.want) {
            const int32_t page = col < n.held ? table[col] : new_page(col);
            if (page >= 0) slot = (int64_t)page * a.page_size + pos % a.page_size;
            if (slot > INT32_MAX) slot = -1;
        }
        a.slots[r.row0 + j] = (int32_t)slot;
        if (a.positions) a.positions[r.row0 + j] = live ? (int32_t)min(pos, (int64_t)INT32_MAX) : -1;
    }
}

// ---- tree_plan --------------------------------------------------------------------
// One warp per request, lane l holds rows l and l + 32.  Pointer doubling: a
// row starts with its own bit and its parent; each of six steps adds the mask
// of the row it points to and moves the pointer there, so the path a mask
// covers doubles and 64 rows are done in 6 steps whatever the tree's depth.
// Bound by the launch: 1.4-1.9 us a call in a replayed graph for one tree, 1.7-2.6 us for
// many (one call a graph, and ten).
constexpr int kTreeWarps = 4;

__global__ void __launch_bounds__(32 * kTreeWarps)
    tree_plan_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ cu_rows,
                     const int32_t* __restrict__ lens, uint64_t* __restrict__ masks, int32_t* __restrict__ positions,
                     int requests, int64_t rows) {
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x * kTreeWarps + (threadIdx.x >> 5);
    const RowRange all = rows_of_all(cu_rows, requests, rows);
    if (b < requests) {
        const PackedRows r = packed_rows(cu_rows, b, all, rows);
        const int n = (int)min(r.n, (int64_t)kTreeMaxRows);
        const int len = max(__ldg(lens + b), 0);
        uint64_t mask[2];
        int up[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            const int p = j < n ? __ldg(parents + r.row0 + j) : -1;
            mask[i] = 1ull << j;
            up[i] = p >= 0 && p < j ? p : -1;
        }
#pragma unroll
        for (int step = 0; step < 6; ++step) {
            uint64_t add[2];
            int next[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int from = up[i] & 31;
                const uint64_t m0 = __shfl_sync(FULL, mask[0], from), m1 = __shfl_sync(FULL, mask[1], from);
                const int u0 = __shfl_sync(FULL, up[0], from), u1 = __shfl_sync(FULL, up[1], from);
                add[i] = up[i] < 0 ? 0 : up[i] < 32 ? m0 : m1;
                next[i] = up[i] < 0 ? -1 : up[i] < 32 ? u0 : u1;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mask[i] |= add[i];
                up[i] = next[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            if (j < n) {
                masks[r.row0 + j] = mask[i];
                positions[r.row0 + j] = (int32_t)min((int64_t)len + __popcll(mask[i]) - 1, (int64_t)INT32_MAX);
            }
        }
        for (int64_t j = kTreeMaxRows + lane; j < r.n; j += 32) {
            masks[r.row0 + j] = 0;
            positions[r.row0 + j] = -1;
        }
    }
    // Rows before the first request and behind the last one.
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    auto clear = [&](int64_t from, int64_t to) {
        for (int64_t j = from + at; j < to; j += step) {
            masks[j] = 0;
            positions[j] = -1;
        }
    };
    clear(0, all.first);
    clear(all.last, rows);
}

// ---- rope_at -----------------------------------------------------------------------
// As rope.cu, with the row's position from the device: a CTA forms the row's (cos, sin)
// table (angle in double), then turns its heads.  Memory-bound: VEC (16-byte
// aligned rows, headDim and rotary_dim / 2 multiples of four) turns four pairs a
// thread with 16-byte accesses: 8111 rows of 40 heads of 128 take 57.6 us, 5.8 TB/s
// (one pair a thread: 70 us).
template <bool VEC>
__global__ void __launch_bounds__(256) rope_at_kernel(const float* x, float* out, int64_t T, int H, int D,
                                                      const int32_t* __restrict__ positions, const RopeDev r) {
    __shared__ __align__(16) float2 cs[kRopeMaxPairs];
    const int half = r.half;
    const int64_t row_len = (int64_t)H * D;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int pos = __ldg(positions + t);
        if (pos < 0) continue;  // the same for every thread of the CTA
        __syncthreads();        // the previous row's table is no longer read
        for (int j = threadIdx.x; j < half; j += blockDim.x) cs[j] = rope_cos_sin(r, pos, j);
        __syncthreads();
        const float* xr = x + t * row_len;
        float* orow = out + t * row_len;
        if constexpr (VEC) {
            const int quads = half / 4;
            for (int e = threadIdx.x; e < H * quads; e += blockDim.x) {
                const int h = e / quads, j = 4 * (e - h * quads);
                const int ia = h * D + (r.interleaved ? 2 * j : j), ib = h * D + (r.interleaved ? 2 * j + 4 : j + half);
                const float4 u = *reinterpret_cast<const float4*>(xr + ia), v = *reinterpret_cast<const float4*>(xr + ib);
                const float4 c01 = *reinterpret_cast<const float4*>(&cs[j]), c23 = *reinterpret_cast<const float4*>(&cs[j + 2]);
                const float2 c0 = make_float2(c01.x, c01.y), c1 = make_float2(c01.z, c01.w), c2 = make_float2(c23.x, c23.y),
                             c3 = make_float2(c23.z, c23.w);
                float4 p, q;
                if (r.interleaved) {
                    p = make_float4(rope_channel(u.x, u.y, true, c0), rope_channel(u.y, u.x, false, c0),
                                    rope_channel(u.z, u.w, true, c1), rope_channel(u.w, u.z, false, c1));
                    q = make_float4(rope_channel(v.x, v.y, true, c2), rope_channel(v.y, v.x, false, c2),
                                    rope_channel(v.z, v.w, true, c3), rope_channel(v.w, v.z, false, c3));
                } else {
                    p = make_float4(rope_channel(u.x, v.x, true, c0), rope_channel(u.y, v.y, true, c1),
                                    rope_channel(u.z, v.z, true, c2), rope_channel(u.w, v.w, true, c3));
                    q = make_float4(rope_channel(v.x, u.x, false, c0), rope_channel(v.y, u.y, false, c1),
                                    rope_channel(v.z, u.z, false, c2), rope_channel(v.w, u.w, false, c3));
                }
                *reinterpret_cast<float4*>(orow + ia) = p;
                *reinterpret_cast<float4*>(orow + ib) = q;
            }
        } else {
            for (int e = threadIdx.x; e < H * half; e += blockDim.x) {
                const int h = e / half, j = e - h * half;
                const int ia = h * D + (r.interleaved ? 2 * j : j);
                const int ib = h * D + (r.interleaved ? 2 * j + 1 : j + half);
                const float a = xr[ia], b = xr[ib];
                orow[ia] = rope_channel(a, b, true, cs[j]);
                orow[ib] = rope_channel(b, a, false, cs[j]);
            }
        }
        if (out != x) {
            const int pass = D - 2 * half;
            for (int e = threadIdx.x; e < H * pass; e += blockDim.x) {
                const int h = e / pass, d = 2 * half + (e - h * pass);
                orow[h * D + d] = xr[h * D + d];
            }
        }
    }
}

// ---- paged_write --------------------------------------------------------------------
// A memory-bound copy: one CTA per packed row at a time, K and V of the row in
// flight together, 16 bytes an access where pointers and widths allow.  A call of
// 514 MB takes 81 us, 6.3 TB/s (94 % of the copy rate); a few rows 1.8 us in a
// replayed graph.
template <typename V>
__global__ void __launch_bounds__(256)
    paged_write_kernel(V* __restrict__ k_pool, V* __restrict__ v_pool, int64_t pool_rows, int64_t kw, int64_t vw,
                       const V* __restrict__ k_new, const V* __restrict__ v_new, const int32_t* __restrict__ slots,
                       int64_t rows) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t slot = __ldg(slots + r);
        if (slot < 0 || slot >= pool_rows) continue;
        for (int64_t i = threadIdx.x; i < kw || i < vw; i += blockDim.x) {
            V a, b;
            if (i < kw) a = __ldcs(k_new + r * kw + i);
            if (i < vw) b = __ldcs(v_new + r * vw + i);
            if (i < kw) k_pool[slot * kw + i] = a;
            if (i < vw) v_pool[slot * vw + i] = b;
        }
    }
}

}  // namespace

cudaError_t launch_page_map(const PageMapArgs& a, cudaStream_t stream) {
    // Chunks of rows per request: enough CTAs for one wave when there are few requests.
    int64_t chunks = (a.rows + kMapThreads - 1) / kMapThreads;
    const int64_t room = kWave / (a.requests + 1);
    if (chunks > room) chunks = room;
    if (chunks < 1) chunks = 1;
    page_map_kernel<<<dim3((unsigned)a.requests + 1, (unsigned)chunks), kMapThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_tree_plan(const int32_t* parents, const int32_t* cu_rows, const int32_t* lens, uint64_t* masks,
                             int32_t* positions, int32_t requests, int64_t rows, cudaStream_t stream) {
    const int64_t blocks = requests > 0 ? ((int64_t)requests + kTreeWarps - 1) / kTreeWarps : 1;
    tree_plan_kernel<<<(unsigned)blocks, 32 * kTreeWarps, 0, stream>>>(parents, cu_rows, lens, masks, positions,
                                                                       requests, rows);
    return cudaGetLastError();
}

cudaError_t launch_rope_at(const float* x, float* out, int64_t T, int H, int D, const int32_t* positions,
                           const RopeDev& r, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    const unsigned blocks = (unsigned)(T < kWave ? T : kWave);
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 && D % 4 == 0 &&
                     r.half % 4 == 0 && r.half > 0;
    if (vec)
        rope_at_kernel<true><<<blocks, 256, 0, stream>>>(x, out, T, H, D, positions, r);
    else
        rope_at_kernel<false><<<blocks, 256, 0, stream>>>(x, out, T, H, D, positions, r);
    return cudaGetLastError();
}

cudaError_t launch_paged_write(float* k_pool, float* v_pool, int64_t pool_rows, int64_t k_width, int64_t v_width,
                               const float* k_new, const float* v_new, const int32_t* slots, int64_t rows,
                               cudaStream_t stream) {
    if (rows == 0 || (k_width == 0 && v_width == 0)) return cudaSuccess;
    const unsigned blocks = (unsigned)(rows < 4 * kWave ? rows : 4 * kWave);
    const uintptr_t mis = reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool) |
                          reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new);
    if ((mis & 15u) == 0 && k_width % 4 == 0 && v_width % 4 == 0)
        paged_write_kernel<float4><<<blocks, 256, 0, stream>>>(
            reinterpret_cast<float4*>(k_pool), reinterpret_cast<float4*>(v_pool), pool_rows, k_width / 4, v_width / 4,
            reinterpret_cast<const float4*>(k_new), reinterpret_cast<const float4*>(v_new), slots, rows);
    else
        paged_write_kernel<float>
            <<<blocks, 256, 0, stream>>>(k_pool, v_pool, pool_rows, k_width, v_width, k_new, v_new, slots, rows);
    return cudaGetLastError();
}

}  // namespace vtmu
