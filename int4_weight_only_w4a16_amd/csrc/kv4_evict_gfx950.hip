// Eviction from the 4-bit key/value cache by accumulated attention weight.
//
// For every sequence and head: with len <= budget slots all are kept; else the
// last `recent` ones and, of the others, the budget - recent with the largest
// weight (equal weights: the lowest slots; the order of the floats' bits with
// -0 as +0, so a NaN counts as larger than anything).  What is kept goes, in
// the order it had, to slots 0 .. of another table's pages: nothing is read
// that the same call writes, so all tiles move at the same time.
//
// select_kernel: a workgroup per sequence and head.  The threshold by a radix
// selection over 11, 11 and 10 bits (a histogram in LDS; integer counts, so the
// order of the adds does not matter): 11 bits first, since the weights' few
// exponents alone would send a wave's adds to a handful of counters.  Then each
// wave counts its part of the slots, and after one exchange of counts writes
// them in order.  Bound by latency: five passes over weights that stay in L2.
// One sequence of 8192 slots, 8 heads: 12.7 us; 16 of 3000 to 33001: 36 us.
// copy_kernel: a workgroup per tile of the destination, all of its loads before the
// first store.  A kept slot whose page is not there becomes NaN, as kv4_read gives it.  Bound
// by the source's cache lines, of which a kept slot's value codes touch
// every one of its tile: 4096 slots of each of those 16 sequences 90 us, 2048 of the one 4.4.

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

// kHeld: groups of 64 weights that a wave keeps in registers through the passes; 0: it reads them
// from memory in each.
template <int kHeld>
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

    constexpr int kBins = 2048, kWaves = kSelect / 64;
    __shared__ __align__(8) unsigned hist[kBins];
    __shared__ unsigned s_bin, s_left;
    __shared__ unsigned counts[kWaves], counts2[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // a part of the slots, whole groups of 64, for each wave
    const int part = ((old + 63) / 64 + kWaves - 1) / kWaves * 64;
    const int from = min(wave * part, old), to = min(from + part, old);
    float held[kHeld > 0 ? kHeld : 8];
    if constexpr (kHeld > 0)
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[j] = acc[min(from + 64 * j + lane, old - 1)];
    // f(slot, weight) for the wave's groups of 64 in order, by all lanes (slots at or past `to` too)
    auto each = [&](auto f) {
        if constexpr (kHeld > 0) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                if (from + 64 * j >= to) break;
                f(from + 64 * j + lane, held[j]);
            }
        } else {
            for (int i0 = from; i0 < to; i0 += 8 * 64) {
#pragma unroll
                for (int j = 0; j < 8; ++j) held[j] = acc[min(i0 + 64 * j + lane, to - 1)];
#pragma unroll
                for (int j = 0; j < 8; ++j) f(i0 + 64 * j + lane, held[j]);
            }
        }
    };
    uint32_t prefix = 0;                         // the threshold's known high bits
    unsigned left = want;                        // how many to take among those with that prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = pass < 2 ? 2047u : 1023u;
        for (int i = threadIdx.x; i < kBins; i += kSelect) hist[i] = 0;
        __syncthreads();
        each([&](int i, float f) {
            const uint32_t k = key_of(f);
            const uint32_t high = pass == 0 ? 0u : pass == 1 ? k >> 21 : k >> 10;
            if (i < to && high == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
        });
        __syncthreads();
        // the bin, counted from the top, in which `left` is reached: thread t has bins 2047 - 2t
        // and 2046 - 2t, a scan over the workgroup the counts above them
        const u2 pair = *reinterpret_cast<const u2 *>(&hist[kBins - 2 - 2 * threadIdx.x]);
        const unsigned h0 = pair[1], h1 = pair[0];
        unsigned run = h0 + h1;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned up = __shfl_up(run, d);
            if (lane >= d) run += up;
        }
        if (lane == 63) counts[wave] = run;
        __syncthreads();
        unsigned above = run - h0 - h1;
#pragma unroll
        for (int j = 0; j < kWaves; ++j) above += j < wave ? counts[j] : 0u;
        if (above < left && above + h0 >= left) {
            s_bin = kBins - 1 - 2 * threadIdx.x;
            s_left = left - above;
        } else if (above + h0 < left && above + h0 + h1 >= left) {
            s_bin = kBins - 2 - 2 * threadIdx.x;
            s_left = left - above - h0;
        }
        __syncthreads();
        prefix = prefix << (pass < 2 ? 11 : 10) | s_bin;
        left = s_left;                           // (written again only after two more barriers)
    }
    // slots above the threshold, and the first `left` equal to it
    const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
    unsigned na = 0, ne = 0;
    each([&](int i, float f) {
        const uint32_t k = key_of(f);
        na += __popcll(__builtin_amdgcn_ballot_w64(i < to && k > prefix));
        ne += __popcll(__builtin_amdgcn_ballot_w64(i < to && k == prefix));
    });
    if (lane == 0) {
        counts[wave] = na;
        counts2[wave] = ne;
    }
    __syncthreads();
    na = ne = 0;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
        na += j < wave ? counts[j] : 0u;
        ne += j < wave ? counts2[j] : 0u;
    }
    each([&](int i, float f) {
        const uint32_t k = key_of(f);
        const bool above = i < to && k > prefix, equal = i < to && k == prefix;
        const uint64_t ma = __builtin_amdgcn_ballot_w64(above), me = __builtin_amdgcn_ballot_w64(equal);
        const unsigned a0 = na + __popcll(ma & below), e0 = ne + __popcll(me & below);
        if (above || (equal && e0 < left)) {
            const unsigned at = a0 + min(e0, left);
            kept[at] = i;
            out[at] = f;
        }
        na += __popcll(ma);
        ne += __popcll(me);
    });
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
    __shared__ uint32_t there_mask;              // bit r32: the slot has a source
    if (threadIdx.x < 64) {
        // (the others take part as slot 0 of the destination: loads without conditions, of which
        // nothing is used)
        const int i = threadIdx.x < 32 ? base + (int)threadIdx.x : len;
        const uint8_t *p = nullptr;
        int s = 0;
        if (i < len) {
            s = a.kept[((int64_t)b * a.c.kv_heads + h) * a.budget + i];
            p = tile_at<D, NG>(a.c, a.c.table, a.c.table_stride, b, h, s >> 5);
        }
        const uint64_t mask = __builtin_amdgcn_ballot_w64(p != nullptr);
        if (threadIdx.x < 32) {
            from[threadIdx.x] = reinterpret_cast<const uint32_t *>(p ? p : dst);
            slot[threadIdx.x] = p ? s & 31 : 0;
        }
        if (threadIdx.x == 0) there_mask = (uint32_t)mask;
    }
    __syncthreads();
    const uint32_t there = there_mask, used = len - base < 32 ? (1u << (len - base)) - 1 : ~0u;
    constexpr uint32_t kNaNs = 0x7FC07FC0u;      // in either type
    uint32_t *words = reinterpret_cast<uint32_t *>(dst);
    constexpr int kCodeWords = T::kCodes / 4;
    constexpr int kKeyWords = 32 * (D / 8) / kCopy, kValueWords = 4 * D / kCopy ? 4 * D / kCopy : 1;
    static_assert(32 * (D / 8) % kCopy == 0, "a whole number of key words a thread");
    uint32_t keys[kKeyWords], values[kValueWords][8];
#pragma unroll
    for (int k = 0; k < kKeyWords; ++k) {
        const int idx = threadIdx.x + k * kCopy, r32 = idx / (D / 8), i = idx % (D / 8);
        keys[k] = from[r32][key_word<D>(slot[r32], i)];
    }
#pragma unroll
    for (int k = 0; k < kValueWords; ++k) {
        const int at = threadIdx.x + k * kCopy, lane = (at >> 2) & 63;
        const int d = 16 * (4 * (at >> 8) + (at & 3)) + (lane & 15);
#pragma unroll
        for (int nib = 0; nib < 8; ++nib) {
            const int r32 = 4 * (lane >> 4) + (nib & 3) + 16 * (nib >> 2);
            values[k][nib] = from[r32][kCodeWords + value_word(slot[r32], d)] >> value_shift(slot[r32]) & 15u;
        }
    }
    uint32_t params[(64 * NG + kCopy - 1) / kCopy];
#pragma unroll
    for (int k = 0; k < (64 * NG + kCopy - 1) / kCopy; ++k) {
        const int at = threadIdx.x + k * kCopy, r32 = at & 31;
        if (at < 64 * NG) params[k] = from[r32][2 * kCodeWords + (at & ~31) + slot[r32]];
    }
#pragma unroll
    for (int k = 0; k < kKeyWords; ++k) {
        const int idx = threadIdx.x + k * kCopy, r32 = idx / (D / 8);
        if (used >> r32 & 1) words[key_word<D>(r32, idx % (D / 8))] = there >> r32 & 1 ? keys[k] : 0u;
    }
#pragma unroll
    for (int k = 0; k < kValueWords; ++k) {
        const int at = threadIdx.x + k * kCopy;
        uint32_t w = 0;
#pragma unroll
        for (int nib = 0; nib < 8; ++nib) {
            const int r32 = 4 * (((at >> 2) & 63) >> 4) + (nib & 3) + 16 * (nib >> 2);
            if (there >> r32 & 1) w |= values[k][nib] << (4 * nib);
        }
        words[kCodeWords + at] = w;
    }
#pragma unroll
    for (int k = 0; k < (64 * NG + kCopy - 1) / kCopy; ++k) {
        const int at = threadIdx.x + k * kCopy;
        if (at < 64 * NG && (used >> (at & 31) & 1))
            words[2 * kCodeWords + at] = there >> (at & 31) & 1 ? params[k] : kNaNs;
    }
}

}  // namespace

hipError_t launch_kv4_evict(const Kv4EvictArgs &a, hipStream_t stream) {
    // weights in registers where those of the longest sequence fit (one sequence of 8192 slots, 8
    // heads: 12.7 us, 14.2 from memory; four times as many spill: 85 us instead of 36)
    const int64_t most = (int64_t)a.max_kv - a.recent;
    const dim3 heads((unsigned)a.c.kv_heads, (unsigned)a.c.batch);
    if (most <= 8 * kSelect)
        select_kernel<8><<<heads, kSelect, 0, stream>>>(a);
    else
        select_kernel<0><<<heads, kSelect, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((a.budget + 31) / 32), (unsigned)a.c.kv_heads, (unsigned)a.c.batch);
    return kv4_dispatch(a.c.head_dim, a.c.groups, [&](auto d, auto ng) {
        copy_kernel<d(), ng()><<<grid, kCopy, 0, stream>>>(a);
        return hipGetLastError();
    });
}

}  // namespace w4a16
