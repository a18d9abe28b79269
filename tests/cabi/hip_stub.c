/*
 * Stand-ins for the runtime calls that a launch makes, so that a test can see
 * what the library would launch without a device: test infrastructure, loaded
 * ahead of the library with its symbols global.
 */
#include <stdint.h>

typedef struct { uint32_t x, y, z; } stub_dim3;

int stub_launches = 0;
uint64_t stub_most_items = 0; /* work-items of the largest launch */

int hipGetDevice(int *device)
{
    *device = 0;
    return 0;
}

/* (The one attribute asked for: compute units.) */
int hipDeviceGetAttribute(int *value, int attribute, int device)
{
    (void)attribute;
    (void)device;
    *value = 256;
    return 0;
}

int hipLaunchKernel(const void *fn, stub_dim3 grid, stub_dim3 block, void **args, uint64_t lds,
                    void *stream)
{
    uint64_t items = (uint64_t)grid.x * grid.y * grid.z * block.x * block.y * block.z;
    (void)fn;
    (void)args;
    (void)lds;
    (void)stream;
    ++stub_launches;
    if (items > stub_most_items)
        stub_most_items = items;
    return items < (1ull << 32) ? 0 : 1; /* hipErrorInvalidValue, as the runtime answers */
}
