// The library's workspaces: one for each (device, stream, slot), grown on demand
// and kept until it is released.  Plain C++: what it asks of the CUDA runtime goes
// through `Api`, so that its failures can be tested without a GPU:
//
//   Stream                                   a stream's handle
//   bool alloc(void **p, size_t n, Stream)   in stream order
//   void free(void *p, Stream)               in stream order
//   bool zero(void *p, size_t n, Stream)     in stream order
//   void release(void *p)                    once nothing runs on the device
//   bool capturing(Stream)                   is the stream being captured into a graph?
//   bool alloc_apart(void **p, size_t n)     in no stream, no part of any capture
//   bool zero_apart(void *p, size_t n)       the same; done when it returns
//
// While its stream is being captured a workspace is allocated apart: allocated in
// stream order it would be the graph's, and the table would hand the graph's
// memory to later calls.  Nor is the one that it replaces freed in stream order
// then.  One that a graph uses stays when a later call needs more: the graph may
// run again.  Both are kept until everything is released.
#pragma once

#include <algorithm>
#include <cstddef>
#include <map>
#include <tuple>
#include <utility>
#include <vector>

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
        const bool apart = api_.capturing(stream);
        if (b.bytes < bytes) {
            if (b.p && (apart || b.graph)) kept_.emplace_back(dev, b.p);
            else if (b.p) api_.free(b.p, stream);
            b = Block{};
            const size_t want = std::max<size_t>(bytes, size_t(1) << 20);
            void *p = nullptr;
            if (!(apart ? api_.alloc_apart(&p, want) : api_.alloc(&p, want, stream))) return SGEMM_ERR_NOMEM;
            if (zeroed && !(apart ? api_.zero_apart(p, want) : api_.zero(p, want, stream))) {
                // (kept, the next call would take it as zeroed)
                if (apart) kept_.emplace_back(dev, p);
                else api_.free(p, stream);
                return SGEMM_ERR_CUDA;
            }
            b = Block{p, want};
        }
        b.graph = b.graph || apart;
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
        for (auto it = kept_.begin(); it != kept_.end();) {
            if (it->first == dev) {
                api_.release(it->second);
                it = kept_.erase(it);
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
        bool graph = false;                      // a graph uses it
    };
    Api api_;
    std::map<Key, Block> blocks_;
    std::vector<std::pair<int, void *>> kept_;   // replaced, but not freed
};

}  // namespace sgemm_gb300
