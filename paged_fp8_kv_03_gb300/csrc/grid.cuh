// Programmatic dependent launches, and sums that keep what rounding loses.
#pragma once

namespace pkv {

// Waits until the kernels ahead in the stream have ended and their writes are
// seen; lets the next kernel be brought onto the GPU (it waits in turn).  What is read
// behind the wait may have been written while this kernel was on the GPU already, so the
// loads are ordinary ones: __ldg() is for memory that nothing writes as long as a kernel lives.
__device__ __forceinline__ void grid_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// a + b rounded, and exactly what that loses (Knuth's two-sum).  Long sums of like
// terms keep it: rounded the same way every time, they drift by up to 2^-24 a term.
__device__ __forceinline__ float two_sum(float a, float b, float &rest)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    rest = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}

}  // namespace pkv
