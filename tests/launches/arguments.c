/* arguments.c - recorder.c that keeps what a kernel is passed too: the first
 * `MOST_BYTES` bytes of each of its first arguments, as many and as long as
 * expect() said for kernels of that name.
 */
#define hipLaunchKernel recorded_launch
#include "recorder.c"
#undef hipLaunchKernel

enum { KINDS = 16, ARGS = 6, MOST_BYTES = 320 };
static struct { char part[64]; int count, size[ARGS]; } kinds[KINDS];
static int known;
static unsigned char kept[MOST][ARGS][MOST_BYTES];

/* Kernels whose name holds `part` take `count` arguments of these sizes. */
void expect(const char* part, int count, const int* size) {
    if (known == KINDS) return;
    strncpy(kinds[known].part, part, sizeof kinds[known].part - 1);
    kinds[known].count = count < ARGS ? count : ARGS;
    for (int i = 0; i < kinds[known].count; ++i) kinds[known].size[i] = size[i] < MOST_BYTES ? size[i] : MOST_BYTES;
    ++known;
}
const unsigned char* argument(int r, int i) { return kept[r][i]; }

int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** args, size_t s, void* st) {
    const int r = count < MOST ? count : MOST - 1;
    recorded_launch(f, g, b, args, s, st);
    for (int k = 0; k < known; ++k)
        if (strstr(records[r].name, kinds[k].part)) {
            for (int i = 0; i < kinds[k].count; ++i) memcpy(kept[r][i], args[i], (size_t)kinds[k].size[i]);
            break;
        }
    return 0;
}
