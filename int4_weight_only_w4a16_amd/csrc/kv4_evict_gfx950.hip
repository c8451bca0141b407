// Eviction from the 4-bit key/value cache by accumulated attention weight.
//
// For every sequence and head: with len <= budget slots all are kept; else the
// last `recent` ones and, of the others, the budget - recent with the largest
// weight (equal weights: the lowest slots; the order of the floats' bits with
// -0 as +0, so a NaN counts as larger than anything).  What is kept goes, in
// the order it had, to slots 0 .. of another table's pages: nothing is read
// that the same call writes, so all tiles move at the same time.
//
// select_kernel: the threshold by a radix selection over eight bits at a time
// (a histogram in LDS, integer counts, so the order of the adds does not
// matter), then the kept slots in order by a scan.  Bound by the passes over
// the weights, which stay in L2.
// copy_kernel: a workgroup per tile of the destination.

#include "kv4_device.hpp"

namespace w4a16 {
namespace {

constexpr int kSelect = 1024;
constexpr int kCopy = 256;

// Unsigned order of the weights' total order.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
    return (u & 0x80000000u) ? ((u & 0x7FFFFFFFu) > 0x7F800000u ? u | 0x80000000u : ~u) : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelect) select_kernel(Kv4EvictArgs a) {
    const int h = blockIdx.x, b = blockIdx.y, kvh = a.c.kv_heads;
    const int64_t cap = (int64_t)a.c.table_stride * a.c.tiles_per_page * 32;
    const int len = (int)min(min((int64_t)min(max(a.kv_len[b], 0), a.max_kv), cap), a.acc_stride);
    const int64_t row = (int64_t)b * kvh + h;
    const float *acc = a.acc + row * a.acc_stride;
    int32_t *kept = a.kept + row * a.budget;
    float *out = a.acc_out + row * a.budget;
    const int keep = min(len, a.budget);
    if (h == 0 && threadIdx.x == 0) a.new_len[b] = keep;
    for (int i = keep + threadIdx.x; i < a.budget; i += kSelect) {
        kept[i] = -1;
        out[i] = 0.f;
    }
    if (len <= a.budget) {
        for (int i = threadIdx.x; i < len; i += kSelect) {
            kept[i] = i;
            out[i] = acc[i];
        }
        return;
    }
    const int old = len - a.recent;              // candidates; more than `want`
    const int want = a.budget - a.recent;
    for (int i = threadIdx.x; i < a.recent; i += kSelect) {
        kept[want + i] = old + i;
        out[want + i] = acc[old + i];
    }
    if (want == 0) return;

    __shared__ unsigned hist[256];
    __shared__ unsigned s_prefix, s_left;
    __shared__ unsigned waves[kSelect / 64];
    uint32_t prefix = 0;                         // the threshold's known high bits
    unsigned left = want;                        // how many to take among those with that prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < old; i += kSelect) {
            const uint32_t k = key_of(acc[i]);
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned n = left;
            int bin = 255;
            while (hist[bin] < n) n -= hist[bin--];      // (the counts above add up to at least `left`)
            s_prefix = prefix << 8 | (unsigned)bin;
            s_left = n;
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
        __syncthreads();
    }
    // slots above the threshold, and the first `left` equal to it
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    unsigned above0 = 0, equal0 = 0;             // counts before this chunk
    for (int i0 = 0; i0 < old; i0 += kSelect) {
        const int i = i0 + threadIdx.x;
        const float f = i < old ? acc[i] : 0.f;
        const uint32_t k = key_of(f);
        const bool above = i < old && k > prefix, equal = i < old && k == prefix;
        const uint64_t ma = __builtin_amdgcn_ballot_w64(above), me = __builtin_amdgcn_ballot_w64(equal);
        const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
        unsigned na = __popcll(ma & below), ne = __popcll(me & below);
        if (lane == 0) waves[wave] = (unsigned)__popcll(ma) | (unsigned)__popcll(me) << 16;
        __syncthreads();
        unsigned all = 0;
        for (int j = 0; j < kSelect / 64; ++j) {
            const unsigned c = waves[j];
            if (j < wave) {
                na += c & 0xFFFFu;
                ne += c >> 16;
            }
            all += c;                            // each half at most 1024
        }
        na += above0;
        ne += equal0;
        if (above || (equal && ne < left)) {
            const unsigned at = na + min(ne, left);
            kept[at] = i;
            out[at] = f;
        }
        above0 += all & 0xFFFFu;
        equal0 += all >> 16;
        __syncthreads();
    }
}

template <int D, int NG>
__global__ void __launch_bounds__(kCopy) copy_kernel(Kv4EvictArgs a) {
    using T = Tile<D, NG>;
    __shared__ const uint32_t *from[32];         // tile of each slot's source
    __shared__ int slot[32];                     // its slot there
    const int tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int len = min(a.new_len[b], a.budget);
    const int base = 32 * tile;
    if (base >= len) return;
    uint8_t *dst = tile_at<D, NG>(a.c, a.dst_table, a.dst_stride, b, h, tile);
    if (!dst) return;
    if (threadIdx.x < 32) {
        const int i = base + threadIdx.x;
        const uint8_t *p = nullptr;
        int s = 0;
        if (i < len) {
            s = a.kept[((int64_t)b * a.c.kv_heads + h) * a.budget + i];
            p = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b, h, s >> 5);
        }
        from[threadIdx.x] = reinterpret_cast<const uint32_t *>(p);
        slot[threadIdx.x] = s & 31;
    }
    __syncthreads();
    uint32_t *words = reinterpret_cast<uint32_t *>(dst);
    for (int idx = threadIdx.x; idx < 32 * (D / 8); idx += kCopy) {
        const int r32 = idx / (D / 8), i = idx % (D / 8);
        if (from[r32]) words[key_word<D>(r32, i)] = from[r32][key_word<D>(slot[r32], i)];
    }
    constexpr int kCodeWords = T::kCodes / 4;
    for (int at = threadIdx.x; at < 4 * D; at += kCopy) {
        const int lane = (at >> 2) & 63;
        const int d = 16 * (4 * (at >> 8) + (at & 3)) + (lane & 15);
        uint32_t w = 0;
#pragma unroll
        for (int nib = 0; nib < 8; ++nib) {
            const int r32 = 4 * (lane >> 4) + (nib & 3) + 16 * (nib >> 2);
            const uint32_t *p = from[r32];
            if (p)
                w |= (p[kCodeWords + value_word(slot[r32], d)] >> value_shift(slot[r32]) & 15u) << (4 * nib);
        }
        words[kCodeWords + at] = w;
    }
    for (int at = threadIdx.x; at < 64 * NG; at += kCopy) {
        const int r32 = at & 31;
        if (from[r32]) words[2 * kCodeWords + at] = from[r32][2 * kCodeWords + (at & ~31) + slot[r32]];
    }
}

}  // namespace

hipError_t launch_kv4_evict(const Kv4EvictArgs &a, hipStream_t stream) {
    select_kernel<<<dim3((unsigned)a.c.kv_heads, (unsigned)a.c.batch), kSelect, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((a.budget + 31) / 32), (unsigned)a.c.kv_heads, (unsigned)a.c.batch);
    return kv4_dispatch(a.c.head_dim, a.c.groups, [&](auto d, auto ng) {
        copy_kernel<d(), ng()><<<grid, kCopy, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace w4a16
