/* Stand-ins for the HIP calls that libtcm.so makes, for tests without a GPU: memory is addresses that nothing touches,
 * and a launch is a line in a log.  Loaded with its symbols global before libtcm.so, whose calls then come here. */
#include <pthread.h>
#include <stdint.h>
#include <string.h>
#include <unistd.h>

typedef struct {
    uint32_t x, y, z;
} dim3;
typedef struct {
    uint64_t thread;
    const void* kernel;
    dim3 grid, block;
} launch_t;

enum { MAX = 1 << 16 };
static launch_t launches[MAX];
static int count, mallocs, pause_us;
static uint64_t next_address = (uint64_t)1 << 45;
static pthread_mutex_t mu = PTHREAD_MUTEX_INITIALIZER;
static __thread struct {
    dim3 grid, block;
    size_t shared;
    void* stream;
} config;

/* the test's side */
int stub_count(void) { return count; }
int stub_mallocs(void) { return mallocs; }
void stub_clear(void) { count = 0; }
void stub_pause(int us) { pause_us = us; } /* after each launch */
const launch_t* stub_launches(void) { return launches; }
uint64_t stub_thread(void) { return (uint64_t)pthread_self(); }

/* the library's */
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) {
    config.grid = grid, config.block = block, config.shared = shared, config.stream = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void** stream) {
    *grid = config.grid, *block = config.block, *shared = config.shared, *stream = config.stream;
    return 0;
}
int hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t shared, void* stream) {
    (void)args, (void)shared, (void)stream;
    pthread_mutex_lock(&mu);
    if (count < MAX) {
        launches[count].thread = (uint64_t)pthread_self();
        launches[count].kernel = kernel;
        launches[count].grid = grid, launches[count].block = block;
        ++count;
    }
    pthread_mutex_unlock(&mu);
    if (pause_us) usleep(pause_us);
    return 0;
}
int hipMalloc(void** p, size_t n) {
    pthread_mutex_lock(&mu);
    *p = (void*)next_address;
    next_address += (n + 4095) & ~(size_t)4095;
    ++mallocs;
    pthread_mutex_unlock(&mu);
    return 0;
}
int hipGetDevice(int* d) { return *d = 0; }
int hipDeviceGetAttribute(int* v, int attribute, int d) {
    (void)attribute, (void)d;
    *v = 256;
    return 0;
}
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int block, size_t shared) {
    (void)f, (void)block, (void)shared;
    *n = 2;
    return 0;
}
int hipStreamIsCapturing(void* stream, int* status) {
    (void)stream;
    return *status = 0;
}
int hipGetSymbolAddress(void** p, const void* symbol) {
    (void)symbol;
    *p = (void*)((uint64_t)1 << 44);
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipFree(void* p) { return (void)p, 0; }
int hipSetDevice(int d) { return (void)d, 0; }
int hipDeviceSynchronize(void) { return 0; }
