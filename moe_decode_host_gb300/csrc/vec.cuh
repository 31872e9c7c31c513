// Loads and stores of short runs of elements whose type (moehost.h: MOE_BF16 ...) is a
// kernel argument: raw bits first, conversion to fp32 later, so that the loads of
// several tensors are in flight together and only the conversions branch on the
// types (uniform branches).
#pragma once

#include <cuda_fp8.h>

#include "internal.cuh"

namespace moe {

__host__ __device__ inline int type_bytes(int t) { return t == MOE_F32 ? 4 : (t == MOE_E4M3 ? 1 : 2); }
inline bool is_float16(int t) { return t == MOE_BF16 || t == MOE_F16; }
inline bool is_float_type(int t) { return is_float16(t) || t == MOE_F32; }

// Whether every run of `vec` elements of a tensor with this base and these strides
// (elements) is aligned to its own size, at most 16 bytes.
inline bool runs_aligned(const void* p, int type, int vec, int64_t s0 = 0, int64_t s1 = 0) {
    const int64_t a = (int64_t)vec * type_bytes(type) < 16 ? (int64_t)vec * type_bytes(type) : 16;
    return reinterpret_cast<uintptr_t>(p) % a == 0 && s0 * type_bytes(type) % a == 0 && s1 * type_bytes(type) % a == 0;
}

namespace {

__device__ __forceinline__ float half_bits_to_f32(uint32_t h, int type) {
    return type == MOE_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
}

// VEC consecutive bf16, f16 or fp32 elements as raw bits.  The loads are plain
// (coherent): outputs may be the inputs' own memory.  WIDE = false: never fp32, half the
// registers.
template <int VEC, bool WIDE = true>
struct Raw {
    uint32_t w[VEC < 2 ? 1 : (WIDE ? VEC : VEC / 2)];

    __device__ __forceinline__ void load(const void* p, int64_t at, int type) {
        if constexpr (VEC == 8) {
            if constexpr (WIDE) if (type == MOE_F32) {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
                const uint4 a = q[0], b = q[1];
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                return;
            }
            {
                const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            }
        } else if constexpr (VEC == 4) {
            if constexpr (WIDE) if (type == MOE_F32) {
                const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
                return;
            }
            {
                const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
                w[0] = a.x, w[1] = a.y;
            }
        } else {
            static_assert(VEC == 1, "runs of 8, 4 or 1");
            w[0] = type == MOE_F32 ? static_cast<const uint32_t*>(p)[at] : static_cast<const uint16_t*>(p)[at];
        }
    }

    // From shared memory: 16-byte pieces `apart` pieces from one another.
    __device__ __forceinline__ void set(const uint4* p, int apart) {
        static_assert(VEC == 8, "runs of 8");
        const uint4 a = p[0];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        if constexpr (WIDE) {
            const uint4 b = p[apart];
            w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
    }

    __device__ __forceinline__ void get(int type, float (&v)[VEC]) const {
        if constexpr (WIDE) if (type == MOE_F32) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(w[i]);
            return;
        }
        if constexpr (VEC == 1) {
            v[0] = half_bits_to_f32(w[0], type);
        } else if (type == MOE_BF16) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Two E4M3 codes, a in the low byte: nearest, ties to even, beyond 448 saturating, NaN kept.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// VEC consecutive elements of type `type`, each rounded once from fp32.
template <int VEC>
__device__ __forceinline__ void store_run(void* p, int64_t at, int type, const float (&v)[VEC]) {
    if (type == MOE_F32) {
        float* q = static_cast<float*>(p) + at;
        if constexpr (VEC == 1) {
            q[0] = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) reinterpret_cast<float4*>(q)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else if (type == MOE_E4M3) {
        uint8_t* q = static_cast<uint8_t*>(p) + at;
        if constexpr (VEC == 1) {
            q[0] = (uint8_t)pack_e4m3(v[0], 0.f);
        } else {
            uint32_t c[VEC / 4];
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i)
                c[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | (pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16);
            if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[1]);
            else *reinterpret_cast<uint32_t*>(q) = c[0];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        if constexpr (VEC == 1) {
            q[0] = (uint16_t)(type == MOE_BF16 ? pack_bf16(v[0], 0.f) : pack_f16(v[0], 0.f));
        } else {
            uint32_t c[VEC / 2];
            if (type == MOE_BF16) {
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) c[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) c[i] = pack_f16(v[2 * i], v[2 * i + 1]);
            }
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(q) = make_uint4(c[0], c[1], c[2], c[3]);
            else *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[1]);
        }
    }
}

}  // namespace
}  // namespace moe
