// rope.cu -- the two ends of a decode step around its attention: queries and
// keys made (RMS norm of each head, position rotation), and new keys and values
// put into a paged cache (keys rotated on the way).
//
// Per head of 128 elements:
//   y = x / sqrt(mean(x^2) + eps) * w                          (w given)
//   pairs (a, b) of the first rot_dim elements -> (a cos t - b sin t,
//   b cos t + a sin t), t = position * inv_freq[i], the pair i being
//   (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved.
//
// Both are streams: each element is read once and written once, with about ten
// operations between, so HBM bounds long calls and the launch bounds short
// ones.  A half-warp holds a head (16 bytes a lane), a warp two heads at a time: the
// norm's sum is four shuffles, and a lane's rotation partners are all in one other
// lane (rot_dim is a multiple of 16).  A warp works on one token, so that nothing
// wider than a warp ever waits: it computes the token's angles once (two a lane; a 64-bit
// product each, since position * inv_freq loses its fraction in 32 bits at far
// positions), keeps them in registers, and goes through the token's heads with
// four pairs of loads in flight.  Few tokens are split by heads over more warps.
// (A CTA of 256 threads that shared the angles of 4 tokens through a barrier, in
// 110 registers, took 72 us where this takes see below: too few warps an SM, all
// of them waiting for the angles.)
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.cuh"

namespace tsa {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopePairs = 4;  // pairs of heads that a warp has in flight

// cos and sin of position * inv_freq.  The product in turns is reduced to
// [-1/2, 1/2] in 64 bits, where positions up to 2^31 keep 20 bits of fraction or more.
__device__ __forceinline__ float2 rope_angle(int pos, double inv_freq) {
    double turns = (double)pos * (inv_freq * 0.15915494309189533577);  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    return make_float2(c, s);
}

// A lane's share of a token's rotation: x[j] -> x[j] * c[j] + partner * s[j].
template <bool INTER>
struct LaneRot {
    float c[8], s[8];
    int src;  // split pairs: the lane (of 32) that holds the partners
    bool on;  // this lane's elements are rotated
    __device__ __forceinline__ void off(int lane) {
        on = false;
        src = lane;
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
    }
    // all lanes; cs: kD / 2 angles of this warp's in shared memory
    __device__ __forceinline__ void load(float2* cs, int pos, const Rotation& rot, int lane) {
        const int half = rot.rot_dim >> 1;
        for (int f = lane; f < half; f += 32) cs[f] = rope_angle(pos, rot.inv_freq[f]);
        __syncwarp();
        const int l = lane & 15, h = rot.rot_dim >> 4;  // lanes of half a rotated head
        if (l >= 2 * h) return;
        on = true;
        if (INTER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = cs[l * 4 + j];
                c[2 * j] = c[2 * j + 1] = v.x;
                s[2 * j] = -v.y;
                s[2 * j + 1] = v.y;
            }
        } else {
            const bool low = l < h;
            src = low ? lane + h : lane - h;
            const int i0 = (low ? l : l - h) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = cs[i0 + j];
                c[j] = v.x;
                s[j] = low ? -v.y : v.y;
            }
        }
    }
    __device__ __forceinline__ void apply(float (&x)[8]) const {  // all lanes
        if (INTER) {
            if (!on) return;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float a = x[j], b = x[j + 1];
                x[j] = fmaf(b, s[j], a * c[j]);
                x[j + 1] = fmaf(a, s[j + 1], b * c[j + 1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = __shfl_sync(0xffffffffu, x[j], src);
                if (on) x[j] = fmaf(p, s[j], x[j] * c[j]);
            }
        }
    }
};

// The heads of one token, two at a time: pairs first, first + step, ... of H heads
// at src + h * sh, through fn(raw) into dst + h * dh.  The first loads are issued
// by the constructor, so that the angles are computed while they are on their way.
struct HeadWalk {
    const uint16_t* src;
    uint16_t* dst;
    long long sh, dh;
    int H, step, h;  // h: this lane's head of the next pair
    uint4 raw[kRopePairs];
    __device__ __forceinline__ HeadWalk(const void* s, long long soff, long long sh_, void* d, long long doff,
                                        long long dh_, int H_, int first, int step_, int lane)
        : sh(sh_), dh(dh_), H(H_), step(2 * step_), h(2 * first + (lane >> 4)) {
        src = static_cast<const uint16_t*>(s) + soff + (lane & 15) * 8;
        dst = static_cast<uint16_t*>(d) + doff + (lane & 15) * 8;
        fetch();
    }
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int u = 0; u < kRopePairs; ++u) {
            const int hu = h + u * step;
            raw[u] = hu < H ? *reinterpret_cast<const uint4*>(src + hu * sh) : make_uint4(0, 0, 0, 0);
        }
    }
    template <class F>
    __device__ __forceinline__ void run(F fn) {
        // (h of the even lanes' head decides for the warp: fn shuffles)
        while (__any_sync(0xffffffffu, h < H)) {
#pragma unroll
            for (int u = 0; u < kRopePairs; ++u) {
                const int hu = h + u * step;
                if (u && !__any_sync(0xffffffffu, hu < H)) break;
                const uint4 y = fn(raw[u]);
                if (hu < H) *reinterpret_cast<uint4*>(dst + hu * dh) = y;
            }
            h += kRopePairs * step;
            fetch();
        }
    }
};

// the place of this warp: token t, the w-th of its W warps; false past the last token
__device__ __forceinline__ bool rope_place(int T, int W, int* t, int* w) {
    const long long i = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    *t = (int)(i / W);
    *w = (int)(i - (long long)*t * W);
    return *t < T;
}

template <class E, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(Heads q, Heads k, Heads qo, Heads ko, int T, int Hq, int Hkv, const float* __restrict__ wq,
                    const float* __restrict__ wk, float eps, const int32_t* __restrict__ positions, Rotation rot, int W) {
    __shared__ float2 cs[kRopeWarps][kD / 2];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    int t, w;
    if (!rope_place(T, W, &t, &w)) return;
    const int pos = rot.rot_dim > 0 ? positions[t] : 0;
    HeadWalk hq(q.p, t * q.st, q.sh, const_cast<void*>(qo.p), t * qo.st, qo.sh, Hq, w, W, lane);
    LaneRot<INTER> lr;
    lr.off(lane);
    if (rot.rot_dim > 0) lr.load(cs[threadIdx.x >> 5], pos, rot, lane);
    auto heads = [&](HeadWalk& hw, const float* weight) {
        float wv[8];
        if (weight) {
            const float4 w0 = *reinterpret_cast<const float4*>(weight + (lane & 15) * 8);
            const float4 w1 = *reinterpret_cast<const float4*>(weight + (lane & 15) * 8 + 4);
            wv[0] = w0.x, wv[1] = w0.y, wv[2] = w0.z, wv[3] = w0.w, wv[4] = w1.x, wv[5] = w1.y, wv[6] = w1.z, wv[7] = w1.w;
        }
        hw.run([&](const uint4& raw) {
            float x[8];
            E::unpack8(raw, x);
            if (weight) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * r * wv[j];
            }
            lr.apply(x);
            return E::pack8(x);
        });
    };
    heads(hq, wq);
    // the keys' pairs go on where the queries' ended, so that the warps share them evenly
    const int pq = (Hq + 1) / 2, fk = (w + W - pq % W) % W;
    HeadWalk hk(k.p, t * k.st, k.sh, const_cast<void*>(ko.p), t * ko.st, ko.sh, Hkv, fk, W, lane);
    heads(hk, wk);
}

template <class E, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
paged_append_kernel(Pages c, Heads k, Heads v, int T, const int32_t* __restrict__ seq, const int32_t* __restrict__ row,
                    const int32_t* __restrict__ positions, Rotation rot, unsigned* __restrict__ flag, int W) {
    __shared__ float2 cs[kRopeWarps][kD / 2];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    int t, w;
    if (!rope_place(T, W, &t, &w)) return;
    // where the token goes: a negative sequence is padding (skipped), anything
    // else out of range sets the flag and is skipped
    const int b = seq ? seq[t] : t, r = row[t], pos = positions ? positions[t] : r;
    if (b < 0) return;
    if (b >= c.B || r < 0 || r >= c.rows_cap()) {
        if (w == 0 && lane == 0) atomicOr(flag, kFlagBounds);
        return;
    }
    const int pg = r / c.page_size;
    const int page = c.table[(long long)b * c.width + pg];
    HeadWalk hk(k.p, t * k.st, k.sh, c.K, 0, c.head_stride, c.Hkv, w, W, lane);
    const int pk = (c.Hkv + 1) / 2, fv = (w + W - pk % W) % W;
    HeadWalk hv(v.p, t * v.st, v.sh, c.V, 0, c.head_stride, c.Hkv, fv, W, lane);
    if (page < 0 || page >= c.num_pages) {
        if (w == 0 && lane == 0) atomicOr(flag, kFlagBounds);
        return;
    }
    const long long at = page * c.page_stride + (long long)(r - pg * c.page_size) * c.row_stride;
    hk.dst += at;
    hv.dst += at;
    hv.run([](const uint4& raw) { return raw; });
    LaneRot<INTER> lr;
    lr.off(lane);
    if (rot.rot_dim > 0) lr.load(cs[threadIdx.x >> 5], pos, rot, lane);
    hk.run([&](const uint4& raw) {
        float x[8];
        E::unpack8(raw, x);
        lr.apply(x);
        return lr.on ? E::pack8(x) : raw;  // unrotated elements bit by bit
    });
}

// Warps of one token: one, unless that leaves the SMs with fewer than 16 each; then
// as many as fill them, a pair of heads each at least.
static int rope_warps(int T, int pairs) {
    const int fill = kPagedSms * 16 / T;
    return fill < 1 ? 1 : fill < pairs ? fill : pairs;
}

template <class... P, class... A>
static cudaError_t rope_launch(void (*kernel)(P...), int T, int W, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)T * W + kRopeWarps - 1) / kRopeWarps));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {pdl_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <class E>
static cudaError_t qk_launch(const Heads& q, const Heads& k, const Heads& qo, const Heads& ko, int T, int Hq, int Hkv,
                             const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
                             const Rotation& rot, cudaStream_t st) {
    const int W = rope_warps(T, (Hq + 1) / 2 + (Hkv + 1) / 2);
    return rope_launch(rot.interleaved ? qk_norm_rope_kernel<E, true> : qk_norm_rope_kernel<E, false>, T, W, st, q, k, qo,
                       ko, T, Hq, Hkv, q_weight, k_weight, eps, positions, rot, W);
}

cudaError_t launch_qk_norm_rope(const Heads& q, const Heads& k, const Heads& qo, const Heads& ko, int T, int Hq, int Hkv,
                                int half, const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const Rotation& rot, cudaStream_t st) {
    if (T == 0 || Hq + Hkv == 0) return cudaSuccess;
    return half ? qk_launch<F16>(q, k, qo, ko, T, Hq, Hkv, q_weight, k_weight, eps, positions, rot, st)
                : qk_launch<Bf16>(q, k, qo, ko, T, Hq, Hkv, q_weight, k_weight, eps, positions, rot, st);
}

template <class E>
static cudaError_t append_launch(const Pages& c, const Heads& k, const Heads& v, int T, const int32_t* seq,
                                 const int32_t* row, const int32_t* positions, const Rotation& rot, unsigned* flag,
                                 cudaStream_t st) {
    const int W = rope_warps(T, 2 * ((c.Hkv + 1) / 2));
    return rope_launch(rot.interleaved ? paged_append_kernel<E, true> : paged_append_kernel<E, false>, T, W, st, c, k, v, T,
                       seq, row, positions, rot, flag, W);
}

cudaError_t launch_paged_append(const Pages& c, const Heads& k, const Heads& v, int T, const int32_t* seq,
                                const int32_t* row, const int32_t* positions, const Rotation& rot, unsigned* flag,
                                cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    return c.half ? append_launch<F16>(c, k, v, T, seq, row, positions, rot, flag, st)
                  : append_launch<Bf16>(c, k, v, T, seq, row, positions, rot, flag, st);
}

}  // namespace tsa
