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
// 110 registers, took 72 us for the first of the cases below.)
//
// Measured (graph replays, a part of the data warm in L2; in brackets calls on inputs that
// are not): 8192 tokens x 40 heads, split pairs (168 MB) 33.8 us = 5.0 TB/s [35.7], where a
// plain copy of those bytes takes 27; 4099 x 72 heads, interleaved (151 MB) 26.9 us [28.6];
// appending 16348 tokens of 8 + 8 heads (134 MB) 22.9 us [24.6]; one token 2.8 us [3.8], a
// launch.  A plain copy of 67 to 84 MB runs at 6.0 to 6.1 TB/s.  Split pairs use 65% of the
// issue slots (140 instructions a pair of heads, the partners' shuffles among them) and
// 43% of HBM.  Walking the heads by pointers instead of indexes took 37.8 and 33.9 us.
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

// A lane's share of a token's rotation and norm weights: x -> x * A + partner * B, two
// elements an instruction, with the weights (of the element, of its partner) in A and B.
template <bool INTER>
struct LaneRot {
    uint64_t A[4], B[4];
    int src;  // split pairs: the lane (of 32) that holds the partners
    bool on;  // this lane's elements are rotated
    float w[8], wp[8];  // the weights of this lane's elements and of their partners (dead once A and B are made)
    __device__ __forceinline__ LaneRot(const Rotation& rot, int lane) {
        const int l = lane & 15, h = rot.rot_dim >> 4;  // h: lanes of half a rotated head
        on = l < 2 * h;
        src = INTER || !on ? lane : l < h ? lane + h : lane - h;
    }
    // the heads' weights [kD], or NULL; requested early
    __device__ __forceinline__ void weights(const float* weight, int lane) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
            const float4 v = weight ? *reinterpret_cast<const float4*>(weight + (lane & 15) * 8 + j) : one;
            w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
            if (!INTER) {
                const float4 p = weight ? *reinterpret_cast<const float4*>(weight + (src & 15) * 8 + j) : one;
                wp[j] = p.x, wp[j + 1] = p.y, wp[j + 2] = p.z, wp[j + 3] = p.w;
            }
        }
    }
    // cs: the token's kD / 2 angles
    __device__ __forceinline__ void coefficients(const float2* cs, const Rotation& rot, int lane) {
        const int l = lane & 15, h = rot.rot_dim >> 4;
        const bool low = l < h;
        const int i0 = INTER ? l * 4 : (low ? l : l - h) * 8;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float2 v[2] = {make_float2(1.f, 0.f), make_float2(1.f, 0.f)};
            if (on) {
                v[0] = cs[INTER ? i0 + j / 2 : i0 + j];
                v[1] = INTER ? v[0] : cs[i0 + j + 1];
            }
            A[j / 2] = pack2(v[0].x * w[j], v[1].x * w[j + 1]);
            // (interleaved: a lane's first of a pair is turned by -sin of the second, the second by sin of the first)
            B[j / 2] = INTER ? pack2(-v[0].y * w[j + 1], v[1].y * w[j])
                             : pack2((low ? -v[0].y : v[0].y) * wp[j], (low ? -v[1].y : v[1].y) * wp[j + 1]);
        }
    }
    __device__ __forceinline__ void apply(uint64_t (&x)[4]) const {  // all lanes
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x0, x1;
            unpack2(x[j], x0, x1);
            uint64_t p;
            if (INTER) {
                p = pack2(x1, x0);
            } else {
                p = pack2(__shfl_sync(0xffffffffu, x0, src), __shfl_sync(0xffffffffu, x1, src));
            }
            x[j] = mul2(x[j], A[j]);
            if (on) x[j] = fma2(p, B[j], x[j]);
        }
    }
};

// the token's angles into this warp's shared memory
__device__ __forceinline__ void token_angles(float2* cs, int pos, const Rotation& rot, int lane) {
    for (int f = lane; f < rot.rot_dim >> 1; f += 32) cs[f] = rope_angle(pos, rot.inv_freq[f]);
    __syncwarp();
}

// The heads of one token, two at a time: pairs first, first + step, ... of H heads
// at src + h * sh, through fn(raw) into dst + h * dh.  The first loads are issued
// by the constructor, so that the angles are computed while they are on their way.
struct HeadWalk {
    const uint16_t* src;
    uint16_t* dst;
    long long sh, dh;
    int H, step, pair, odd;  // pair: the next one (the whole warp's); odd: this half-warp's head of a pair
    uint4 raw[kRopePairs];
    __device__ __forceinline__ HeadWalk(const void* s, long long soff, long long sh_, void* d, long long doff,
                                        long long dh_, int H_, int first, int step_, int lane)
        : H(H_), step(step_), pair(first), odd(lane >> 4) {
        src = static_cast<const uint16_t*>(s) + soff + odd * sh_ + (lane & 15) * 8;
        dst = static_cast<uint16_t*>(d) + doff + odd * dh_ + (lane & 15) * 8;
        sh = 2 * sh_;
        dh = 2 * dh_;
        fetch();
    }
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int u = 0; u < kRopePairs; ++u) {
            const int p = pair + u * step;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (2 * p + odd < H) raw[u] = *reinterpret_cast<const uint4*>(src + p * sh);
        }
    }
    template <class F>
    __device__ __forceinline__ void run(F fn) {  // all lanes together: fn shuffles
        while (2 * pair < H) {
#pragma unroll
            for (int u = 0; u < kRopePairs; ++u) {
                const int p = pair + u * step;
                if (u && 2 * p >= H) break;
                const uint4 y = fn(raw[u]);
                if (2 * p + odd < H) *reinterpret_cast<uint4*>(dst + p * dh) = y;
            }
            pair += kRopePairs * step;
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

// The kernel before may write any input (a decode loop advances its positions and rows on
// the device) and may still run when this one starts.  So the inputs are plain pointers: as
// __restrict__ to const they would be taken for unchanged while the kernel runs, and the
// compiler could read them ahead of the wait, or through the cache that is not coherent.
template <class E, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(Heads q, Heads k, Heads qo, Heads ko, int T, int Hq, int Hkv, const float* wq,
                    const float* wk, float eps, const int32_t* positions, Rotation rot, int W) {
    __shared__ float2 cs[kRopeWarps][kD / 2];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    int t, w;
    if (!rope_place(T, W, &t, &w)) return;
    const int pos = rot.rot_dim > 0 ? positions[t] : 0;
    HeadWalk hq(q.p, t * q.st, q.sh, const_cast<void*>(qo.p), t * qo.st, qo.sh, Hq, w, W, lane);
    LaneRot<INTER> lr(rot, lane);
    lr.weights(wq, lane);
    token_angles(cs[threadIdx.x >> 5], pos, rot, lane);
    auto heads = [&](HeadWalk& hw, const float* weight) {
        lr.coefficients(cs[threadIdx.x >> 5], rot, lane);
        hw.run([&](const uint4& raw) {
            uint64_t x[4];
            E::unpack8(raw, x);
            float r = 1.f;
            if (weight) {
                uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
                for (int j = 1; j < 4; ++j) sq = fma2(x[j], x[j], sq);
                float s0, s1;
                unpack2(sq, s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
            }
            lr.apply(x);
            if (weight) {
                const uint64_t rr = pack2(r, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], rr);
            }
            return E::pack8(x);
        });
    };
    heads(hq, wq);
    lr.weights(wk, lane);
    // the keys' pairs go on where the queries' ended, so that the warps share them evenly
    const int pq = (Hq + 1) / 2, fk = (w + W - pq % W) % W;
    HeadWalk hk(k.p, t * k.st, k.sh, const_cast<void*>(ko.p), t * ko.st, ko.sh, Hkv, fk, W, lane);
    heads(hk, wk);
}

template <class E, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
paged_append_kernel(Pages c, Heads k, Heads v, int T, const int32_t* seq, const int32_t* row,
                    const int32_t* positions, Rotation rot, unsigned* flag, int W) {
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
    token_angles(cs[threadIdx.x >> 5], pos, rot, lane);
    LaneRot<INTER> lr(rot, lane);
    lr.weights(nullptr, lane);
    lr.coefficients(cs[threadIdx.x >> 5], rot, lane);
    hk.run([&](const uint4& raw) {
        uint64_t x[4];
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
