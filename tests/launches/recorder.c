/* recorder.c - a stand-in for the HIP runtime that notes what a library asks it
 * for (kernel launches and function attributes) and runs nothing, so that launch
 * shapes of any size can be looked at on a machine without a GPU.  Test
 * infrastructure: load it with RTLD_GLOBAL before the library.
 */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3_t;
typedef struct {
    char name[160];   /* the kernel's (mangled) */
    uint32_t grid[3], block[3];
    uint64_t lds;     /* dynamic bytes of a launch, or the attribute's value */
    int32_t launch;   /* 1: a launch, 0: an attribute */
} record_t;

enum { MOST = 4096 };
static record_t records[MOST];
static int count;
static struct { const void* f; const char* name; } names[MOST];
static int named;
static dim3_t grid, block;
static size_t lds;
static void* stream;

int recorded(void) { return count; }
const record_t* record(int i) { return &records[i]; }
void forget(void) { count = 0; }

static record_t* add(const void* f) {
    record_t* r = &records[count < MOST ? count++ : MOST - 1];
    memset(r, 0, sizeof *r);
    for (int i = 0; i < named; ++i)
        if (names[i].f == f) strncpy(r->name, names[i].name, sizeof r->name - 1);
    return r;
}

void** __hipRegisterFatBinary(const void* data) { static void* p; (void)data; return &p; }
void __hipUnregisterFatBinary(void** m) { (void)m; }
void __hipRegisterFunction(void** m, const void* f, char* d, const char* name, unsigned n, void* a, void* b, void* c,
                           void* e, int* w) {
    (void)m; (void)d; (void)n; (void)a; (void)b; (void)c; (void)e; (void)w;
    if (named < MOST) { names[named].f = f; names[named++].name = name; }
}
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t s, void* st) {
    grid = g; block = b; lds = s; stream = st;
    return 0;
}
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* s, void** st) {
    *g = grid; *b = block; *s = lds; *st = stream;
    return 0;
}
int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** args, size_t s, void* st) {
    (void)args; (void)st;
    record_t* r = add(f);
    memcpy(r->grid, &g, sizeof g);
    memcpy(r->block, &b, sizeof b);
    r->lds = s;
    r->launch = 1;
    return 0;
}
int hipFuncSetAttribute(const void* f, int attr, int value) {
    (void)attr;
    add(f)->lds = (uint64_t)value;
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int attr, int d) { (void)attr; (void)d; *v = 0; return 0; }
