// The table of workspaces against a CUDA runtime of its own that writes down what it is
// asked, and fails where it is told to.  Prints what went wrong, or nothing.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

#include "../dense_fp32_gemm_05_gb300/csrc/workspace.h"

using namespace sgemm_gb300;

#define CHECK(x)                                                     \
    do {                                                             \
        if (!(x)) {                                                  \
            std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x);     \
            std::exit(1);                                            \
        }                                                            \
    } while (0)

struct State {
    std::map<void *, size_t> live;
    std::map<void *, bool> zeros;
    std::map<void *, bool> apart;       // not allocated in stream order
    bool alloc_fails = false, zero_fails = false, capturing = false;
    int allocs = 0;
};
static State g;

struct Fake {
    using Stream = int;
    bool capturing(Stream) { return g.capturing; }
    bool alloc_apart(void **p, size_t n) {
        if (!take(p, n)) return false;
        g.apart[*p] = true;
        return true;
    }
    // in stream order: a node of the graph, while the stream is captured
    bool alloc(void **p, size_t n, Stream) {
        CHECK(!g.capturing);
        return take(p, n);
    }
    bool take(void **p, size_t n) {
        if (g.alloc_fails) return false;
        *p = reinterpret_cast<void *>(static_cast<size_t>(0x1000 * ++g.allocs));
        g.live[*p] = n;
        return true;
    }
    void free(void *p, Stream) {
        CHECK(!g.capturing && !g.apart[p]);
        CHECK(g.live.erase(p) == 1);
    }
    bool zero(void *p, size_t n, Stream) {
        CHECK(!g.capturing && !g.apart[p]);
        return clear(p, n);
    }
    bool zero_apart(void *p, size_t n) {
        CHECK(g.apart[p]);
        return clear(p, n);
    }
    bool clear(void *p, size_t n) {
        CHECK(g.live.count(p) && g.live[p] >= n);
        if (g.zero_fails) return false;
        g.zeros[p] = true;
        return true;
    }
    void release(void *p) { CHECK(g.live.erase(p) == 1); }
};

static void reuse_and_growth() {
    Workspaces<Fake> w;
    void *a = nullptr, *b = nullptr;
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK && g.live[a] >= 100);
    CHECK(w.get(0, 1, 0, 200, false, &b) == SGEMM_OK && b == a);          // a megabyte at least
    CHECK(w.get(0, 1, 0, 3 << 20, false, &b) == SGEMM_OK && b != a && !g.live.count(a));
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK && a == b);
    void *other[3];
    CHECK(w.get(0, 2, 0, 100, false, &other[0]) == SGEMM_OK);            // another stream, slot, device
    CHECK(w.get(0, 1, 1, 100, false, &other[1]) == SGEMM_OK);
    CHECK(w.get(1, 1, 0, 100, false, &other[2]) == SGEMM_OK);
    CHECK(g.live.size() == 4);
    w.release(0);
    CHECK(g.live.size() == 1 && g.live.count(other[2]));
    w.release(1);
    CHECK(g.live.empty());
}

static void an_allocation_fails() {
    Workspaces<Fake> w;
    void *a = nullptr;
    g.alloc_fails = true;
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_ERR_NOMEM);
    g.alloc_fails = false;
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK && g.live.size() == 1);
    g.alloc_fails = true;
    CHECK(w.get(0, 1, 0, 2 << 20, false, &a) == SGEMM_ERR_NOMEM);
    g.alloc_fails = false;
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK && g.live.size() == 1);
}

static void zeroing_fails() {
    // counters that were never zeroed are not handed to the next call
    Workspaces<Fake> w;
    void *a = nullptr;
    g.zero_fails = true;
    CHECK(w.get(0, 1, 3, 256, true, &a) == SGEMM_ERR_CUDA);
    CHECK(g.live.empty());
    CHECK(w.get(0, 1, 3, 256, true, &a) == SGEMM_ERR_CUDA);
    g.zero_fails = false;
    CHECK(w.get(0, 1, 3, 256, true, &a) == SGEMM_OK && g.zeros[a]);
    g.zeros.clear();
    CHECK(w.get(0, 1, 3, 256, true, &a) == SGEMM_OK && g.zeros.empty());   // (zeroed once)
}

static void a_stream_that_is_captured() {
    // a cold stream: nothing becomes the graph's, and calls after the capture take the same
    Workspaces<Fake> w;
    void *a = nullptr, *b = nullptr, *c = nullptr;
    g.capturing = true;
    CHECK(w.get(0, 1, 3, 256, true, &a) == SGEMM_OK && g.apart[a] && g.zeros[a]);
    CHECK(w.get(0, 1, 0, 100, false, &b) == SGEMM_OK && g.apart[b]);
    g.capturing = false;
    CHECK(w.get(0, 1, 3, 256, true, &c) == SGEMM_OK && c == a);
    CHECK(w.get(0, 1, 0, 100, false, &c) == SGEMM_OK && c == b);
    w.release(0);
    CHECK(g.live.empty());
    // a warm one that has to grow: the old memory may be in use before the capture
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK && !g.apart[a]);
    g.capturing = true;
    CHECK(w.get(0, 1, 0, 2 << 20, false, &b) == SGEMM_OK && b != a && g.live.count(a) && g.apart[b]);
    g.zero_fails = true;
    CHECK(w.get(0, 1, 3, 256, true, &c) == SGEMM_ERR_CUDA);
    g.zero_fails = false;
    CHECK(w.get(0, 1, 3, 256, true, &c) == SGEMM_OK && g.zeros[c]);
    g.capturing = false;
    w.release(0);
    CHECK(g.live.empty());
}

static void growth_after_a_capture() {
    // the memory that a captured call uses outlives a larger call on its stream
    Workspaces<Fake> w;
    void *a = nullptr, *b = nullptr, *c = nullptr;
    CHECK(w.get(0, 1, 0, 100, false, &a) == SGEMM_OK);                    // allocated before the capture
    g.capturing = true;
    CHECK(w.get(0, 1, 0, 100, false, &b) == SGEMM_OK && b == a);
    g.capturing = false;
    CHECK(w.get(0, 1, 0, 2 << 20, false, &b) == SGEMM_OK && b != a && g.live.count(a));
    CHECK(w.get(0, 1, 0, 4 << 20, false, &c) == SGEMM_OK && c != b && !g.live.count(b));   // (no graph's)
    g.capturing = true;
    CHECK(w.get(0, 1, 0, 8 << 20, false, &b) == SGEMM_OK && g.apart[b]);  // allocated under it
    g.capturing = false;
    CHECK(w.get(0, 1, 0, 16 << 20, false, &c) == SGEMM_OK && g.live.count(b) && g.live.count(a));
    w.release(0);
    CHECK(g.live.empty());
}

int main(int, char **argv) {
    const std::string what = argv[1];
    if (what == "reuse_and_growth") reuse_and_growth();
    else if (what == "an_allocation_fails") an_allocation_fails();
    else if (what == "zeroing_fails") zeroing_fails();
    else if (what == "a_stream_that_is_captured") a_stream_that_is_captured();
    else if (what == "growth_after_a_capture") growth_after_a_capture();
    else return 2;
    return 0;
}
