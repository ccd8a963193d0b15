"""The build's check of register counts, on what ptxas prints."""
import pytest

from decode_attention_compressed_gb300 import build as B

SAID = """ptxas info    : 0 bytes gmem, 4 bytes cmem[4]
ptxas info    : Compiling entry function '_ZN2zf12_GLOBAL__N_115q4_chunk_kernelILi3EEEvNS_9ChunkArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN2zf12_GLOBAL__N_115q4_chunk_kernelILi3EEEvNS_9ChunkArgsE
    8 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2zf12_GLOBAL__N_120q4_chunk_join_kernelENS_9ChunkArgsEi' for 'sm_103a'
ptxas info    : Used 31 registers, used 0 barriers
"""


def test_a_kernel_with_other_registers_fails_the_build():
    B.check_registers(SAID.format(96))
    for count in (88, 95, 97, 104):
        with pytest.raises(RuntimeError, match=f"q4_chunk_kernel.*{count} registers"):
            B.check_registers(SAID.format(count))
    B.check_registers("")


def test_only_the_named_kernels_are_checked():
    B.check_registers(SAID.format(50), want={"other_kernel": 96})
    with pytest.raises(RuntimeError, match="q4_chunk_join_kernel"):
        B.check_registers(SAID.format(50), want={"q4_chunk_join_kernel": 32})
