// Queries and keys normalised for each head and rotated by their positions
// (gdn_qk_norm), and the gradients (gdn_qk_norm_backward).  Per token and head,
//
//     n = r x,  z = w n,  y = scale R z,   r = rsqrt(c sum x^2 + eps)
//     dz = scale R^T dy,  dw = sum dz n,  dx = r (w dz - n c <w dz, n>)
//
// with c = 1 (L2) or 1 / d (RMS).  Six operations for an element read and
// written (14 in the backward pass, for two read and one written): bound by HBM.
//
// d / 8 lanes of a wave share a head, 8 channels each, so a wave takes 4 or 8
// heads side by side and the sums stay within 16 lanes.  A lane's channels are
// those that its rotation pairs: 4 from the first half of the rotated channels and
// their partners from the second, or 8 neighbours, so nothing is exchanged for the
// rotation.  The angles of a token are the same for all its heads: a lane forms
// its four once and goes through the heads, two loads at a time.
//
// Measured, bf16 (a copy reaches 5.1 TB/s, and 5.95 where it overwrites its input):
// unit vectors of 65,536 tokens of 64 heads of 128 channels, 2.147 GB in 361 to 373 us,
// 5.8 TB/s, and no byte moves twice (FETCH_SIZE and WRITE_SIZE 1.074 GB each).
// Gradients of 32,768 tokens of 40 heads with weights and rotation, 1.007 GB in 180 to
// 189 us, 5.5 TB/s, of which the weights' sums are 4.5.  64 tokens take 3.8 us, about an
// empty launch.  fp32: 32,768 tokens of 40 heads with weights and rotation, 1.342 GB in
// 240 us, 5.6 TB/s; of 64 heads without rotation, where a lane's two loads take every second
// 16 bytes each, 2.147 GB in 474, 4.5.  Heads in steps of one load or four, and half or twice as many
// workgroups, are slower or the same.  Tensors that the caches cannot hold are read
// and written past them: 380 us where it was 406, the gradients 189 where it was 200.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_lanes.h"
#include "gdn_stack_kernels.h"

namespace gdn {
namespace {

constexpr int kWaves = 4;         // of a workgroup
template <bool BACK>
constexpr int kUnroll = BACK ? 1 : 2;  // steps of heads whose loads are in flight together
constexpr int64_t kUnits = 8192;  // waves' worth of work from which on a wave takes all heads of a token
constexpr int64_t kCaches = 256 << 20;
constexpr int64_t kMostBlocks = 1024;  // of the backward pass: partial sums of the weights' gradients

enum Rotation { kNone, kHalves, kPairs };

struct Norm {
    const void *x[2], *dy[2];
    int64_t stride[2], out_stride[2];
    void* out[2];
    const float* weight[2];
    float* partial;  // [workgroup][2][d] sums of the weights' gradients, or NULL
    int32_t heads[2];
    int64_t T;
    bool norm;
    float c, eps;
    const int32_t* positions;
    const float* freq;
    int32_t rotary;
    float scale[2];
    int32_t per;       // waves that share a token
    int32_t steps[2];  // of heads, for a token
};

// Sum over the D / 8 lanes of a head; every lane receives it.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
    if constexpr (D == 128) return across<Sum, 1, 8>(x);
    auto moved = [](float y, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(y), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    x += moved(x, std::integral_constant<int, 0xb1>{});   // lanes 1 apart within four
    x += moved(x, std::integral_constant<int, 0x4e>{});   // 2 apart
    x += moved(x, std::integral_constant<int, 0x141>{});  // mirrored within eight
    return x;
}

// A lane's two groups of four channels, and the angles that turn them.
template <int D, int ROT>
struct Lane {
    int group, c0, c1, f;
    bool turns;
    float cs[4], sn[4];
    __device__ __forceinline__ Lane(const Norm& a) {
        const int lane = threadIdx.x & 63, l = lane % (D / 8);
        group = lane / (D / 8);
        turns = ROT != kNone && 8 * l < a.rotary;
        c0 = ROT == kHalves && turns ? 4 * l : 8 * l;
        c1 = ROT == kHalves && turns ? a.rotary / 2 + 4 * l : 8 * l + 4;
        f = 4 * l;
    }
    // Whole turns are taken off in 64 bits: an angle may be a million radians.
    __device__ __forceinline__ void angles(const Norm& a, int64_t t) {
        if (ROT == kNone || !turns) return;
        const double p = a.positions[t];
        const floatx4 freq = *reinterpret_cast<const floatx4*>(a.freq + f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double x = p * ((double)freq[j] * 0.15915494309189533577);
            sincospif(2.f * (float)(x - rint(x)), &sn[j], &cs[j]);
        }
    }
    // The lane's channels turned by its angles; SIGN -1: back.
    template <int SIGN>
    __device__ __forceinline__ void turn(float* v) const {
        if (ROT == kNone || !turns) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = ROT == kHalves ? j : 2 * j, q = ROT == kHalves ? j + 4 : 2 * j + 1;
            const float u = v[p], w = v[q], s = SIGN * sn[j];
            v[p] = u * cs[j] - w * s;
            v[q] = u * s + w * cs[j];
        }
    }
};

// A lane's eight values, in one load where they are neighbours of two bytes.
// PASSING: by the caches, for a call whose tensors are far larger than these.
template <typename V, bool PASSING>
__device__ __forceinline__ V load(const void* at) {
    const V* const p = static_cast<const V*>(at);
    if constexpr (PASSING) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool PASSING, typename V>
__device__ __forceinline__ void store(void* at, V x) {
    V* const p = static_cast<V*>(at);
    if constexpr (PASSING) __builtin_nontemporal_store(x, p);
    else *p = x;
}
template <typename T, int ROT, bool PASSING>
struct Eight {
    static constexpr bool ONE = sizeof(T) == 2 && ROT != kHalves;
    typedef T four __attribute__((ext_vector_type(4)));
    typedef T eight __attribute__((ext_vector_type(8)));
    eight v;
    __device__ __forceinline__ void load8(const T* at, int c0, int c1) {
        if constexpr (ONE) {
            v = load<eight, PASSING>(at + c0);
        } else {
            const four a = load<four, PASSING>(at + c0), b = load<four, PASSING>(at + c1);
            v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    __device__ __forceinline__ static void store8(T* at, int c0, int c1, const float* x) {
        eight y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = from_f32<T>(x[j]);
        if constexpr (ONE) {
            store<PASSING>(at + c0, y);
        } else {
            store<PASSING>(at + c0, __builtin_shufflevector(y, y, 0, 1, 2, 3));
            store<PASSING>(at + c1, __builtin_shufflevector(y, y, 4, 5, 6, 7));
        }
    }
};

// One step: the D / 8 lanes of each head at `head` of kind s, of token t.
template <typename T, int D, int ROT, bool BACK, bool PASSING>
struct Step {
    Eight<T, ROT, PASSING> in, back;
    __device__ __forceinline__ void load(const Norm& a, const Lane<D, ROT>& l, int s, int64_t t, int32_t head) {
        head = head < a.heads[s] ? head : 0;  // lanes without a head work on the first, unseen
        in.load8(static_cast<const T*>(a.x[s]) + t * a.stride[s] + head * D, l.c0, l.c1);
        if (BACK) back.load8(static_cast<const T*>(a.dy[s]) + (t * a.heads[s] + head) * D, l.c0, l.c1);
    }
    __device__ __forceinline__ void store(const Norm& a, const Lane<D, ROT>& l, int s, int64_t t, int32_t head, const float* w,
                                          float* dw) {
        const bool live = head < a.heads[s];
        float x[8], r = 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_f32(in.v[j]);
        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += x[j] * x[j];
            r = __builtin_amdgcn_rsqf(head_sum<D>(sum) * a.c + a.eps);  // good to one step of fp32
        }
        float v[8];
        if (!BACK) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = x[j] * r * w[j];
            l.template turn<1>(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= a.scale[s];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = to_f32(back.v[j]) * a.scale[s];
                x[j] *= r;
            }
            l.template turn<-1>(v);
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (live) dw[j] += v[j] * x[j];
                v[j] *= w[j];
                dot += v[j] * x[j];
            }
            if (a.norm) {
                dot = head_sum<D>(dot) * a.c;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r * (v[j] - x[j] * dot);
            }
        }
        if (live) in.store8(static_cast<T*>(a.out[s]) + t * a.out_stride[s] + head * D, l.c0, l.c1, v);
    }
};

template <typename T, int D, int ROT, bool BACK, bool PASSING>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_kernel(Norm a) {
    constexpr int HEADS = 64 / (D / 8);  // of a step
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Lane<D, ROT> l(a);
    float w[2][8], dw[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[s][j] = a.weight[s] ? a.weight[s][j < 4 ? l.c0 + j : l.c1 + j - 4] : 1.f;
            dw[s][j] = 0.f;
        }
    const int64_t units = a.T * a.per;
    for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < units; u += (int64_t)gridDim.x * kWaves) {
        const int64_t t = u / a.per;
        const int32_t part = (int32_t)(u - t * a.per);
        const int32_t all = a.steps[0] + a.steps[1];
        const int32_t from = (int32_t)((int64_t)all * part / a.per), to = (int32_t)((int64_t)all * (part + 1) / a.per);
        l.angles(a, t);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            int32_t i = s == 0 ? from : (from > a.steps[0] ? from - a.steps[0] : 0);
            const int32_t end = s == 0 ? (to < a.steps[0] ? to : a.steps[0]) : to - a.steps[0];
            for (; i + kUnroll<BACK> <= end; i += kUnroll<BACK>) {
                Step<T, D, ROT, BACK, PASSING> step[kUnroll<BACK>];
#pragma unroll
                for (int k = 0; k < kUnroll<BACK>; ++k) step[k].load(a, l, s, t, (i + k) * HEADS + l.group);
#pragma unroll
                for (int k = 0; k < kUnroll<BACK>; ++k) step[k].store(a, l, s, t, (i + k) * HEADS + l.group, w[s], dw[s]);
            }
            for (; i < end; ++i) {
                Step<T, D, ROT, BACK, PASSING> step;
                step.load(a, l, s, t, i * HEADS + l.group);
                step.store(a, l, s, t, i * HEADS + l.group, w[s], dw[s]);
            }
        }
    }
    if (BACK && a.partial) {
        __shared__ float sums[kWaves * HEADS][2][D];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[wave * HEADS + l.group][s][j < 4 ? l.c0 + j : l.c1 + j - 4] = dw[s][j];
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += 64 * kWaves) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < kWaves * HEADS; ++k) sum += sums[k][i / D][i % D];
            a.partial[(int64_t)blockIdx.x * 2 * D + i] = sum;
        }
    }
}

// The weights' gradients from the workgroups' sums: a workgroup for four channels
// of one kind, in an order that their number alone decides.
struct WeightSums {
    const float* partial;
    float* out[2];
    int32_t blocks, d;
};
__global__ __launch_bounds__(256) void weight_sums_kernel(WeightSums a) {
    __shared__ floatx4 sums[256];
    const int per = a.d / 4, s = blockIdx.x / per, c = blockIdx.x % per * 4;
    if (!a.out[s]) return;
    floatx4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int b = threadIdx.x; b < a.blocks; b += 256)
        sum += *reinterpret_cast<const floatx4*>(a.partial + ((int64_t)b * 2 + s) * a.d + c);
    sums[threadIdx.x] = sum;
    __syncthreads();
#pragma unroll
    for (int n = 128; n > 0; n /= 2) {
        if ((int)threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) *reinterpret_cast<floatx4*>(a.out[s] + c) = sums[0];
}

int64_t steps_of(int32_t heads, int32_t d) { return (heads + 512 / d - 1) / (512 / d); }

// Waves that share a token: one where tokens fill the device, else as many as
// there are steps of heads.
int64_t waves_per_token(int64_t T, int64_t steps) {
    return std::max<int64_t>(1, std::min<int64_t>(steps, T > 0 ? kUnits / T : 1));
}
int64_t backward_blocks(int64_t T, int32_t H, int32_t H_k, int32_t d) {
    const int64_t units = T * waves_per_token(T, steps_of(H, d) + steps_of(H_k, d));
    return std::min((units + kWaves - 1) / kWaves, kMostBlocks);
}

Norm arguments(const QkNormLaunch& p) {
    Norm a = {};
    for (int s = 0; s < 2; ++s) {
        a.x[s] = p.x[s]; a.dy[s] = p.dy[s];
        a.stride[s] = p.stride[s]; a.out_stride[s] = p.out_stride[s];
        a.out[s] = p.out[s];
        a.weight[s] = p.weight[s];
        a.heads[s] = p.heads[s];
        a.steps[s] = (int32_t)steps_of(p.heads[s], p.d);
    }
    a.T = p.T;
    a.norm = p.norm != 0;
    a.c = p.norm == 2 ? 1.f / (float)p.d : 1.f;
    a.eps = p.eps;
    a.positions = p.positions;
    a.freq = p.inv_freq;
    a.rotary = p.rotary;
    a.scale[0] = p.q_scale;
    a.scale[1] = 1.f;
    a.per = (int32_t)waves_per_token(p.T, a.steps[0] + a.steps[1]);
    return a;
}

template <bool BACK, bool PASSING, typename T, int D>
void run_rotation(const Norm& a, const QkNormLaunch& p, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(64 * kWaves);
    if (p.rotary == 0) hipLaunchKernelGGL((qk_norm_kernel<T, D, kNone, BACK, PASSING>), grid, block, 0, s, a);
    else if (p.interleaved) hipLaunchKernelGGL((qk_norm_kernel<T, D, kPairs, BACK, PASSING>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((qk_norm_kernel<T, D, kHalves, BACK, PASSING>), grid, block, 0, s, a);
}
// Outputs that the caches cannot hold pass them by (1.1 GB: 370 us, through them
// 406); smaller ones stay for whoever reads them next.
template <bool BACK, typename T, int D>
void run_size(const Norm& a, const QkNormLaunch& p, unsigned blocks, hipStream_t s) {
    if (p.T * ((int64_t)p.heads[0] + p.heads[1]) * D * (int64_t)sizeof(T) > kCaches) run_rotation<BACK, true, T, D>(a, p, blocks, s);
    else run_rotation<BACK, false, T, D>(a, p, blocks, s);
}
template <bool BACK>
hipError_t run(const Norm& a, const QkNormLaunch& p, int64_t blocks, hipStream_t s) {
    if (p.bf16 && p.d == 128) run_size<BACK, bf16, 128>(a, p, (unsigned)blocks, s);
    else if (p.bf16) run_size<BACK, bf16, 64>(a, p, (unsigned)blocks, s);
    else if (p.d == 128) run_size<BACK, float, 128>(a, p, (unsigned)blocks, s);
    else run_size<BACK, float, 64>(a, p, (unsigned)blocks, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm(const QkNormLaunch& p, hipStream_t s) {
    const Norm a = arguments(p);
    if (p.T == 0 || a.steps[0] + a.steps[1] == 0) return hipSuccess;
    // (grids of less than 2^24 workgroups: what is more takes another turn)
    return run<false>(a, p, std::min<int64_t>((p.T * a.per + kWaves - 1) / kWaves, 1 << 23), s);
}

size_t qk_norm_backward_workspace_bytes(int64_t T, int32_t H, int32_t H_k, int32_t d) {
    return (size_t)backward_blocks(T, H, H_k, d) * 2 * (size_t)d * sizeof(float);
}

hipError_t launch_qk_norm_backward(const QkNormLaunch& p, hipStream_t s) {
    Norm a = arguments(p);
    const bool sums = p.d_weight[0] || p.d_weight[1];
    const int64_t blocks = a.steps[0] + a.steps[1] == 0 ? 0 : backward_blocks(p.T, p.heads[0], p.heads[1], p.d);
    if (sums) a.partial = static_cast<float*>(p.workspace);
    if (blocks > 0) {
        const hipError_t e = run<true>(a, p, blocks, s);
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    const WeightSums w = {a.partial, {p.d_weight[0], p.d_weight[1]}, (int32_t)blocks, p.d};
    hipLaunchKernelGGL(weight_sums_kernel, dim3(2 * p.d / 4), dim3(256), 0, s, w);
    return hipGetLastError();
}

}  // namespace gdn
