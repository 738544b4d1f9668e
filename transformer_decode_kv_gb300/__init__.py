"""GB300-native (sm_103a) decode library for Llama-architecture GQA transformers with a KV cache.

The product is the C-ABI shared library libllm.so (include/llm.h, sources in csrc/); this package
holds its sources, its build script and a thin ctypes binding with the same call names.
"""
from .binding import (AttnPlan, Context, KvPages, LlmError, lib, kv_load, kv_store,  # noqa: F401
                      sample_rows, F32, F16, BF16, F8_E4M3, Q8_0, LIB_PATH, SIGNATURES)
