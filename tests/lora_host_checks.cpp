// CPU driver for the overlap checks of the dense layers' operators at spans past 2^32 bytes (moe_layer_host.cpp), built
// without HIP under the address and undefined-behaviour sanitizers by tests/test_lora_sanitized.py.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "../mixture_experts_fp8_amd/csrc/moe_layer_plan.h"

using namespace moe;

#define CHECK(cond)                                                                                   \
    do {                                                                                              \
        if (!(cond)) {                                                                                \
            std::fprintf(stderr, "%s:%d: CHECK(%s) failed; last error: %s\n", __FILE__, __LINE__, #cond, \
                         host::last_error());                                                         \
            std::exit(1);                                                                             \
        }                                                                                             \
    } while (0)
#define REFUSED(call, text) CHECK((call) == MOE_ERR_INVALID && std::strstr(host::last_error(), text))

// buffers 8 GiB apart, never dereferenced
template <typename T>
static T* at(int i) { return reinterpret_cast<T*>((uintptr_t)0x10000000u + ((uintptr_t)i << 33)); }

// The most adapters that a count holds: a is 7.4 TB (864 places less a little), b 4.9 TB (576 places).
static moe_lora_args many_adapters() {
    moe_lora_args l{};
    l.T = 6, l.K = 72, l.N = 48, l.R = 24, l.num_adapters = 2147483647, l.num_seqs = 6, l.x = at<uint16_t>(0), l.ld_x = 80;
    l.y = at<float>(1), l.ld_y = 96, l.workspace = at<void>(2), l.workspace_bytes = lora_plan(6, 24, 0, false).end;
    l.adapter_ids = at<int32_t>(3), l.scale = at<float>(4), l.a = at<uint16_t>(10), l.b = at<uint16_t>(1000);
    return l;
}

int main() {
    moe_lora_args l = many_adapters();
    CHECK(host::check_lora(&l) == MOE_OK);
    for (int place : {10, 81, 800, 873}) {   // in a, the last one in its last 8 GiB
        l = many_adapters();
        l.y = at<float>(place);
        REFUSED(host::check_lora(&l), "y must not overlap a");
        l = many_adapters();
        l.workspace = at<void>(place);
        REFUSED(host::check_lora(&l), "workspace must not overlap a");
    }
    for (int place : {1000, 1100, 1575}) {   // in b
        l = many_adapters();
        l.y = at<float>(place);
        REFUSED(host::check_lora(&l), "y must not overlap b");
        l = many_adapters();
        l.workspace = at<void>(place);
        REFUSED(host::check_lora(&l), "workspace must not overlap b");
    }
    for (int place : {874, 900, 1576, 2000}) {   // between them and behind
        l = many_adapters();
        l.y = at<float>(place);
        CHECK(host::check_lora(&l) == MOE_OK);
        l = many_adapters();
        l.workspace = at<void>(place);
        CHECK(host::check_lora(&l) == MOE_OK);
    }
    l = many_adapters();   // scale: 8 GiB of floats less one
    l.y = reinterpret_cast<char*>(at<float>(5)) - 256;
    REFUSED(host::check_lora(&l), "y must not overlap scale");

    // the most rows, far apart: x is 281 TB, y and the residual are 2^20 elements apart (35 TB of float32)
    l = many_adapters();
    l.num_adapters = 3, l.a = at<uint16_t>(1), l.b = at<uint16_t>(2), l.scale = nullptr;
    l.T = 1 << 23, l.num_seqs = 1, l.seq_offsets = at<int32_t>(4), l.workspace = at<void>(5);
    l.workspace_bytes = lora_plan(1 << 23, 24, 1, false).end;
    CHECK(l.workspace_bytes < (size_t)1 << 33);
    l.x = at<uint16_t>(100), l.ld_x = 1 << 24, l.y = at<float>(40000), l.ld_y = 1 << 20;
    CHECK(host::check_lora(&l) == MOE_OK);
    l.y = at<float>(32867);                  // x ends with the place before 100 + 32768
    REFUSED(host::check_lora(&l), "y must not overlap x");
    l.y = at<float>(32868);
    CHECK(host::check_lora(&l) == MOE_OK);
    l.ld_x = (1 << 24) + 8;
    CHECK(host::check_lora(&l) == MOE_ERR_UNSUPPORTED);
    l.ld_x = 1 << 24, l.y = at<float>(40000), l.ld_residual = 1 << 20;
    l.residual = at<float>(40001);           // whole rows further: the same columns
    REFUSED(host::check_lora(&l), "y must not overlap residual");
    l.residual = at<float>(40001) + 48;      // other columns of rows that y has too
    CHECK(host::check_lora(&l) == MOE_OK);
    l.residual = at<float>(40001) + 40;
    REFUSED(host::check_lora(&l), "y must not overlap residual");
    l.residual = at<float>(44096);           // behind y's last row
    CHECK(host::check_lora(&l) == MOE_OK);

    // the gated block's outputs of many rows: h 68 GB, gu twice that
    moe_gated_linear_args f{};
    f.T = 8000000, f.K = 128, f.I = 4160, f.xq = at<uint8_t>(0), f.xs = at<uint8_t>(1), f.w = at<uint8_t>(2), f.w_scale = at<uint8_t>(3);
    f.h = at<uint16_t>(100), f.gu = at<uint16_t>(200);
    CHECK(host::check_gated_linear(&f) == MOE_OK);
    f.gu = at<uint16_t>(107);
    CHECK(host::check_gated_linear(&f) == MOE_ERR_INVALID);
    f.gu = at<uint16_t>(108);
    CHECK(host::check_gated_linear(&f) == MOE_OK);
    f.gu = at<uint16_t>(85);
    CHECK(host::check_gated_linear(&f) == MOE_ERR_INVALID);
    f.xq = at<uint8_t>(107), f.gu = nullptr;
    REFUSED(host::check_gated_linear(&f), "h must not overlap xq");
    std::puts("lora host checks ok");
    return 0;
}
