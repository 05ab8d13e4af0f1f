// The library's workspaces: one for each (device, stream, slot), grown on demand
// and kept until it is released.  Plain C++: what it asks of the CUDA runtime goes
// through `Api`, so that its failures can be tested without a GPU:
//
//   Stream                                   a stream's handle
//   bool alloc(void **p, size_t n, Stream)   in stream order
//   void free(void *p, Stream)               in stream order
//   bool zero(void *p, size_t n, Stream)     in stream order
//   void release(void *p)                    once nothing runs on the device
#pragma once

#include <algorithm>
#include <cstddef>
#include <map>
#include <tuple>

#include "../../include/sgemm_gb300.h"

namespace sgemm_gb300 {

template <typename Api>
class Workspaces {
public:
    using Stream = typename Api::Stream;

    explicit Workspaces(Api api = Api()) : api_(api) {}

    // At least `bytes` private to (device, stream, slot); with `zeroed`, zeros when it
    // is new.
    int get(int dev, Stream stream, int slot, size_t bytes, bool zeroed, void **out) {
        Block &b = blocks_[Key{dev, stream, slot}];
        if (b.bytes < bytes) {
            if (b.p) api_.free(b.p, stream);
            b = Block{};
            const size_t want = std::max<size_t>(bytes, size_t(1) << 20);
            void *p = nullptr;
            if (!api_.alloc(&p, want, stream)) return SGEMM_ERR_NOMEM;
            if (zeroed && !api_.zero(p, want, stream)) {
                api_.free(p, stream);            // (kept, the next call would take it as zeroed)
                return SGEMM_ERR_CUDA;
            }
            b = Block{p, want};
        }
        *out = b.p;
        return SGEMM_OK;
    }

    // Everything of a device, on which nothing runs.
    void release(int dev) {
        for (auto it = blocks_.begin(); it != blocks_.end();) {
            if (std::get<0>(it->first) == dev) {
                if (it->second.p) api_.release(it->second.p);
                it = blocks_.erase(it);
            } else {
                ++it;
            }
        }
    }

    Api &api() { return api_; }

private:
    using Key = std::tuple<int, Stream, int>;
    struct Block {
        void *p = nullptr;
        size_t bytes = 0;
    };
    Api api_;
    std::map<Key, Block> blocks_;
};

}  // namespace sgemm_gb300
