// recorder.cpp -- the HIP calls that libreduce makes, without a GPU.
//
// Loaded with global symbols before libreduce.so, these functions take the
// place of the runtime's.  Memory is addresses that nothing looks at; a kernel
// launch is checked against the runtime's limit of 2^32 - 1 work-items and
// counted.  So a test on the CPU sees what a call of any size would launch.
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <new>

namespace {
struct Dim3 {
    uint32_t x, y, z;
};
int last_error = 0;
uint64_t launches = 0, largest = 0, allocated = 0, freed = 0;
uintptr_t next_address = uintptr_t(1) << 46;
bool out_of_host_memory = false;
constexpr int kInvalidConfiguration = 9;

// The launch shape between <<<>>> and the kernel's host function.
struct {
    Dim3 grid, block;
    std::size_t lds;
    void* stream;
} pending;

uint64_t volume(const Dim3& d) { return (uint64_t)d.x * d.y * d.z; }
} // namespace

// Host allocations of the library fail while out_of_host_memory is set.
void* operator new(std::size_t n)
{
    void* p = out_of_host_memory ? nullptr : std::malloc(n ? n : 1);
    if (!p)
        throw std::bad_alloc();
    return p;
}

extern "C" {
int hipGetDevice(int* device)
{
    *device = 0;
    return 0;
}
int hipDeviceGetAttribute(int* value, int, int)
{
    *value = 256; // compute units
    return 0;
}
int hipGetLastError()
{
    const int e = last_error;
    last_error = 0;
    return e;
}
int hipMalloc(void** p, std::size_t n)
{
    *p = reinterpret_cast<void*>(next_address);
    next_address += (n + 4095) / 4096 * 4096;
    ++allocated;
    return 0;
}
int hipFree(void*)
{
    ++freed;
    return 0;
}
int hipStreamSynchronize(void*) { return 0; }
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, std::size_t lds, void* stream)
{
    pending = {grid, block, lds, stream};
    return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, std::size_t* lds, void** stream)
{
    *grid = pending.grid;
    *block = pending.block;
    *lds = pending.lds;
    *stream = pending.stream;
    return 0;
}
int hipLaunchKernel(const void*, Dim3 grid, Dim3 block, void**, std::size_t, void*)
{
    const uint64_t items = volume(grid) * volume(block);
    ++launches;
    largest = items > largest ? items : largest;
    if (items == 0 || items >> 32 || volume(block) > 1024)
        last_error = kInvalidConfiguration;
    return last_error;
}

uint64_t recorded_launches() { return launches; }
uint64_t recorded_largest() { return largest; }
uint64_t recorded_allocations() { return allocated; }
uint64_t recorded_frees() { return freed; }
void record_from_here() { launches = largest = allocated = freed = 0; }
void set_out_of_host_memory(int on) { out_of_host_memory = on != 0; }
}
