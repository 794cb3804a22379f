// Products of the gated block's backward pass, bf16 operands.
#include "prod_api.hpp"
#include "prod_launch.hpp"

#define TG_PLAIN(OT)                                                                                           \
    template <>                                                                                                \
    hipError_t tg::launch_plain_two<1, OT>(const ProdArgs &p0, const PlainEpi<1> &e0, const ProdArgs &p1,      \
                                           const PlainEpi<OT> &e1, hipStream_t s) {                            \
        return launch_prod_two<1>(p0, e0, p1, e1, s);                                                          \
    }
TG_PLAIN(0)
TG_PLAIN(1)
