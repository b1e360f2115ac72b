// The kernels of qmm_gemv.hip with an epilogue before the store (qmm_epilogue.h).
#define QMM_WITH_EPILOGUE
#include "qmm_gemv.hip"
