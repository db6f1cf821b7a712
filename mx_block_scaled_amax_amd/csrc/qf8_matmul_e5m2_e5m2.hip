// qf8_matmul_e5m2_e5m2.hip -- the matrix products of E5M2 rows with E5M2 columns.
#include "qf8_matmul.h"

namespace qf8 {
template int launch_matmul_formats<kE5M2, kE5M2>(const MatmulArgs &, int, int, int, int64_t, hipStream_t);
}
