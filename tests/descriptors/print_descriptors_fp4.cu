// Prints the 4-bit MMA's instruction descriptors (host-side evaluation of the
// encoder the kernel calls), one per line: <name> <argument...> <value>.  Read
// by tests/test_descriptors_fp4.py.
#include <cstdint>
#include <cstdio>
#include "ptx_fp4.cuh"

using namespace fp8bs;

int main()
{
    const uint32_t shapes[][2] = {{128, 16}, {128, 32}, {128, 64}, {128, 128}, {128, 256}, {256, 256}};
    for (const auto& s : shapes)
        for (uint32_t id = 0; id < 4; id += 2)
            std::printf("idesc_e2m1_bs %u %u %u %u\n", s[0], s[1], id, idesc_e2m1_bs(s[0], s[1], id));
    return 0;
}
