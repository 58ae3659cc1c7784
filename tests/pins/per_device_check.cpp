// What is done once on each device: again on another device, again after a failure, and not otherwise.
#include <cstdio>

#include "../../block_scaled_fp4_amax_amd/csrc/per_device.h"

int main()
{
    fp4q::OncePerDevice once;
    int calls = 0, status = 0;
    const auto set = [&] { ++calls; return status; };
    struct { int device, status, want, calls; } steps[] = {
        {0, 0, 0, 1}, {0, 7, 0, 1}, {1, 7, 7, 2}, {1, 7, 7, 3}, {1, 0, 0, 4}, {1, 7, 0, 4}, {63, 0, 0, 5}, {63, 7, 0, 5},
        {0, 7, 0, 5}, {64, 0, 0, 6}, {64, 0, 0, 7}, {2, 0, 0, 8}};
    for (auto& s : steps) {
        status = s.status;
        if (once(s.device, set) != s.want || calls != s.calls) {
            std::printf("device %d: %d calls\n", s.device, calls);
            return 1;
        }
    }
    std::printf("ok\n");
    return 0;
}
