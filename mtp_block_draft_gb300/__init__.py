"""GB300-native (sm_103a) DMTP speculative-decoding round.

The round lives in the C-ABI library ``libdmtp.so`` (include/dmtp.h; the draft-depth
gate in include/dmtp_gate.h; the draft heads' token list in include/dmtp_vocab.h; the
operators of a decode step over a paged cache in include/dmtp_ops.h); this package holds
its CUDA sources (``csrc/``), the in-tree build (``build.py``) and the ctypes binding
(``binding.py``; of the operators, ``ops.py``).
"""
from .binding import (DmtpError, DmtpGate, DmtpRound, DmtpVocabList, default_max_ctx,
                      load_library, make_config, make_weights)
from .ops import DmtpPagedCache, add_rmsnorm_e4m3, sample_rows

__all__ = ["DmtpError", "DmtpGate", "DmtpPagedCache", "DmtpRound", "DmtpVocabList",
           "add_rmsnorm_e4m3", "default_max_ctx", "load_library", "make_config", "make_weights",
           "sample_rows"]
