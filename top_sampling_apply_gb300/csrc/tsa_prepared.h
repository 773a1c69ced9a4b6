// What has been set on the kernels (dynamic shared memory, cluster size), by
// kernel and device.  No CUDA here: a host compiler takes this file alone.
#pragma once
#include <stddef.h>

#include <new>

namespace tsa {

struct Prepared {
    const void *fn;
    int device;
    size_t smem;
    int cluster16;
};

// Grows as kernels and devices come, in blocks, so that entries stay where they
// are.  The caller holds a lock.
class PreparedTable {
  public:
    // The entry of a kernel on a device, with nothing set if it is new; NULL if
    // there is no memory for one.
    Prepared *find(const void *fn, int device) {
        for (Block *b = &first_;; b = b->next) {
            for (int i = 0; i < b->used; ++i)
                if (b->entry[i].fn == fn && b->entry[i].device == device) return &b->entry[i];
            if (b->used < kBlock) {
                b->entry[b->used] = Prepared{fn, device, 0, 0};
                return &b->entry[b->used++];
            }
            if (!b->next) b->next = new (std::nothrow) Block();
            if (!b->next) return nullptr;
        }
    }

  private:
    static constexpr int kBlock = 64;
    struct Block {
        Prepared entry[kBlock];
        int used = 0;
        Block *next = nullptr;
    };
    Block first_;
};

}  // namespace tsa
