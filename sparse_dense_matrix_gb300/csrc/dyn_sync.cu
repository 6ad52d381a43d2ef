// What becomes of a bounded wait that gave up in a call whose pattern is chosen at run
// time. These calls have no handle that could carry an error word: each stream gets
// words of its own when it first launches one of the kernels that wait (past kSlots
// streams, some share theirs). A launch that is captured writes to slot 0, as a graph may
// be replayed on any stream.
// So that nobody's failure is taken away by somebody else's question, a set word is
// moved into its slot's count of failures, and a stream is answered by what that count
// was when it was last told: it hears of each failure of its own slot and of the graphs'
// once. (It may so hear of the failure of a graph that ran elsewhere; none misses its own.)
#include <mutex>
#include <new>
#include <unordered_map>

#include "dyn.cuh"

namespace spmm {
namespace {

constexpr int kSlots = 256, kMaxDevices = 64;    // slot 0: captured launches
constexpr int kErrTaken = kErrTimeout + 2;       // of a slot's kErrWords words
static_assert(kErrTaken < kErrWords, "a word for the exchange");

__device__ int32_t g_dynamic_err[kSlots * kErrWords];

__global__ void k_take_words(int32_t *err, int slot) {
    int32_t *e = err + (threadIdx.x ? slot : 0) * kErrWords;
    e[kErrTaken] = atomicExch(e + kErrTimeout, 0);
}

struct Stream {
    int slot = 0;                                // 0: no launch of its own was seen
    uint64_t own = 0, graphs = 0;                // failures that it was told of
};

struct Device {
    uint64_t failures[kSlots] = {};
    int next_slot = 1;
    std::unordered_map<const void *, Stream> streams;
};

struct State {
    std::mutex lock;
    Device device[kMaxDevices];
};

State *state() {
    static State *s = new (std::nothrow) State;  // never destroyed: calls may come late
    return s;
}

cudaError_t current_device(int *dev) {
    if (!state()) return cudaErrorMemoryAllocation;
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    return *dev < kMaxDevices ? cudaSuccess : cudaErrorNotSupported;
}

}  // namespace

cudaError_t dynamic_err(cudaStream_t s, int32_t **err) {
    int dev = 0, slot = 0;
    cudaStreamCaptureStatus capturing;
    cudaError_t e = cudaGetSymbolAddress((void **)err, g_dynamic_err);
    if (e == cudaSuccess) e = current_device(&dev);
    if (e == cudaSuccess) e = cudaStreamIsCapturing(s, &capturing);
    if (e != cudaSuccess) return e;
    if (capturing == cudaStreamCaptureStatusNone) {
        std::lock_guard<std::mutex> hold(state()->lock);
        Device &d = state()->device[dev];
        try {
            Stream &me = d.streams[s];
            if (!me.slot) {
                me.slot = d.next_slot;
                me.own = d.failures[me.slot];
                d.next_slot = d.next_slot % (kSlots - 1) + 1;
            }
            slot = me.slot;
        } catch (const std::bad_alloc &) {       // slot 0 then: told to all
        }
    }
    *err += slot * kErrWords;
    return cudaSuccess;
}

}  // namespace spmm

extern "C" spmm_status spmm_dynamic_sync(void *stream) {
    using namespace spmm;
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    int32_t *err = nullptr, words[kSlots * kErrWords];
    cudaError_t e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = current_device(&dev);
    if (e == cudaSuccess) e = cudaGetSymbolAddress((void **)&err, g_dynamic_err);
    if (e != cudaSuccess) return cuda_status(e);
    std::lock_guard<std::mutex> hold(state()->lock);
    Device &d = state()->device[dev];
    Stream me;
    const auto known = d.streams.find(s);
    if (known != d.streams.end()) me = known->second;
    const auto read = [&](int word) {
        cudaError_t r = cudaMemcpyAsync(words, err, sizeof(words), cudaMemcpyDeviceToHost, s);
        if (r == cudaSuccess) r = cudaStreamSynchronize(s);
        if (r != cudaSuccess) return r;
        for (const int slot : {0, me.slot})
            words[slot * kErrWords] = words[slot * kErrWords + word];
        return r;
    };
    e = read(kErrTimeout);
    if (e == cudaSuccess && (words[0] || words[me.slot * kErrWords])) {
        // moved out in one step: a failure that comes after it is the next one
        k_take_words<<<1, me.slot ? 2 : 1, 0, s>>>(err, me.slot);
        count_launch();
        e = cudaGetLastError();
        if (e == cudaSuccess) e = read(kErrTaken);
        if (e == cudaSuccess) {
            if (words[0]) ++d.failures[0];
            if (me.slot && words[me.slot * kErrWords]) ++d.failures[me.slot];
        }
    }
    if (e != cudaSuccess) return cuda_status(e);
    const bool told = me.graphs != d.failures[0] || (me.slot && me.own != d.failures[me.slot]);
    if (!told) return SPMM_OK;
    me.graphs = d.failures[0];
    if (me.slot) me.own = d.failures[me.slot];
    try {
        d.streams[s] = me;
    } catch (const std::bad_alloc &) {           // told again the next time
    }
    return SPMM_ERR_TIMEOUT;
}
