// Reordering of beam states in place: beam w of item b continues the state of
// beam parents[b][w], over the item's first lengths[b] positions.
//
// A unit (1 to 16 bytes, the widest that the pointers, strides and positions
// allow) at one place of the state depends on the units at the same place of
// the item's other beams only: one thread reads them all and then writes the
// ones that changed, so no second buffer and no order between threads is
// needed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kThreads = 256;
constexpr int kStatesPerLaunch = 64;

struct StateList {
    char* p[kStatesPerLaunch];
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <class U, int W>
__global__ void __launch_bounds__(kThreads)
    reorder_kernel(StateList list, int w_n, const int32_t* __restrict__ parents, int64_t beam_stride,
                   int64_t outer_stride, int64_t n_positions, int64_t position_bytes,
                   const int32_t* __restrict__ lengths) {
    const int64_t item = blockIdx.y;
    // blockIdx.z: state, blockIdx.x: outer x chunk, see the launcher
    const int64_t chunks = gridDim.x;
    int64_t n = n_positions;
    if (lengths) {
        const int64_t l = lengths[item];
        n = l < 0 ? 0 : l < n ? l : n;
    }
    const int64_t units = n * (position_bytes / static_cast<int64_t>(sizeof(U)));
    const int32_t* pa = parents + item * w_n;
    char* base = list.p[blockIdx.z % kStatesPerLaunch] + (blockIdx.z / kStatesPerLaunch) * outer_stride +
                 item * w_n * beam_stride;
    int src[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        src[w] = w;
        if (w < w_n) {
            const int p = pa[w];
            if (p >= 0 && p < w_n) src[w] = p;
        }
    }
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < units; i += chunks * kThreads) {
        U v[W];
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (src[w] != w) v[w] = *reinterpret_cast<const U*>(base + src[w] * beam_stride + i * sizeof(U));
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (src[w] != w) *reinterpret_cast<U*>(base + w * beam_stride + i * sizeof(U)) = v[w];
    }
}

template <class U, int W>
hipError_t launch_shape(const ReorderArgs& a, int64_t item, int n_items, int state, int n_states, int64_t outer,
                        hipStream_t s) {
    StateList list{};
    for (int k = 0; k < n_states; ++k)
        list.p[k] = static_cast<char*>(a.states[state + k]) + outer * a.outer_stride + item * a.n_beams * a.beam_stride;
    const int64_t units = a.n_positions * (a.position_bytes / static_cast<int64_t>(sizeof(U)));
    int64_t x = (units + kThreads - 1) / kThreads;
    if (x > 1024) x = 1024;
    reorder_kernel<U, W><<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(n_items),
                                static_cast<unsigned>(n_states)), kThreads, 0, s>>>(
        list, a.n_beams, a.parents + item * a.n_beams, a.beam_stride, a.outer_stride, a.n_positions, a.position_bytes,
        a.lengths ? a.lengths + item : nullptr);
    return hipGetLastError();
}

template <class U>
hipError_t launch_beams(const ReorderArgs& a, int64_t item, int n_items, int state, int n_states, int64_t outer,
                        hipStream_t s) {
    if (a.n_beams <= 4) return launch_shape<U, 4>(a, item, n_items, state, n_states, outer, s);
    if (a.n_beams <= 16) return launch_shape<U, 16>(a, item, n_items, state, n_states, outer, s);
    return launch_shape<U, 64>(a, item, n_items, state, n_states, outer, s);
}

}  // namespace

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t stream) {
    uint64_t bits = static_cast<uint64_t>(a.position_bytes);
    if (a.n_items * a.n_beams > 1) bits |= static_cast<uint64_t>(a.beam_stride);
    if (a.n_outer > 1) bits |= static_cast<uint64_t>(a.outer_stride);
    for (int k = 0; k < a.n_states; ++k) bits |= reinterpret_cast<uintptr_t>(a.states[k]);
    for (int k = 0; k < a.n_states; k += kStatesPerLaunch)
        for (int64_t o = 0; o < a.n_outer; ++o)
            for (int64_t b = 0; b < a.n_items; b += 32768) {
                const int ns = a.n_states - k < kStatesPerLaunch ? a.n_states - k : kStatesPerLaunch;
                const int nb = static_cast<int>(a.n_items - b < 32768 ? a.n_items - b : 32768);
                hipError_t e;
                if (bits % 4 == 0) e = launch_beams<uint32_t>(a, b, nb, k, ns, o, stream);
                else if (bits % 2 == 0) e = launch_beams<uint16_t>(a, b, nb, k, ns, o, stream);
                else e = launch_beams<uint8_t>(a, b, nb, k, ns, o, stream);
                if (e != hipSuccess) return e;
            }
    return hipSuccess;
}

}  // namespace kldk
