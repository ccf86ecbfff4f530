// Test-only kernel: the experts' sigmoid and silu of every fp32 number against 64 bits. Built by the test that uses it; not part
// of the library.
#include "ep_expert_tiles.cuh"

namespace {

// worst[0], worst[1]: the largest error of the sigmoid (as its two factors) and of silu relative to themselves, as the bits of a
// double; worst[2]: numbers whose silu is NaN, infinite or 0 where the definition's is not, or the other way round.
__global__ void sigmoid_sweep_kernel(unsigned long long* worst) {
    double sigmoid_off = 0.0, silu_off = 0.0;
    unsigned long long wrong = 0;
    for (uint64_t i = blockIdx.x * static_cast<uint64_t>(blockDim.x) + threadIdx.x; i < (uint64_t{1} << 32); i += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
        const float v = __uint_as_float(static_cast<uint32_t>(i));
        const ep::Sigmoid s = ep::sigmoid_of(v);
        const double got = static_cast<double>(s.r) * (s.far ? 0x1p-124 : 1.0), want = 1.0 / (1.0 + exp(-static_cast<double>(v)));
        const float gate = ep::gated(v, 1.0f);
        const double silu = static_cast<double>(v) * want;
        if (v != v || silu != silu) {   // NaN and -infinity
            if (gate == gate) ++wrong;
            continue;
        }
        if (want >= 0x1p-249) sigmoid_off = fmax(sigmoid_off, fabs(got - want) / want);
        else if (!(got >= 0.0 && got < 0x1p-248)) ++wrong;
        if (isinf(silu) || isinf(gate)) {
            if (static_cast<double>(gate) != silu) ++wrong;
        } else {   // (half a step of the subnormal numbers)
            silu_off = fmax(silu_off, fmax(fabs(gate - silu) - 0x1p-150, 0.0) / fmax(fabs(silu), 0x1p-300));
        }
    }
    atomicMax(worst, static_cast<unsigned long long>(__double_as_longlong(sigmoid_off)));
    atomicMax(worst + 1, static_cast<unsigned long long>(__double_as_longlong(silu_off)));
    atomicAdd(worst + 2, wrong);
}

}  // namespace

// worst: three 64-bit numbers on the device, zeros.
extern "C" int sigmoid_sweep(void* worst, void* stream) {
    sigmoid_sweep_kernel<<<152 * 8, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<unsigned long long*>(worst));
    return cudaGetLastError() == cudaSuccess ? 0 : 1;
}
